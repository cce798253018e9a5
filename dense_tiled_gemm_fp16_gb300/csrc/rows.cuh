// Rows of 16-bit values, eight a lane and 256 a warp: loads and stores of rows that
// start at any element.
#pragma once

#include "mxf4_format.cuh"

namespace row_dev {

template <int kValue>
struct Int {
    static constexpr int value = kValue;
};

using mxf4_dev::Elem;

// Sixteen bytes from byte `o` (0, 2, .. 14) of 32, `o` the same in a warp: a branch on the
// word and four shifts, a third of what selecting them takes.
__device__ __forceinline__ void take16(const uint32_t* in, uint32_t o, uint32_t* out)
{
    const uint32_t bits = (o & 2u) * 8u;
    auto from = [&](auto k) {
#pragma unroll
        for (int c = 0; c < 4; ++c) out[c] = __funnelshift_r(in[k.value + c], in[k.value + c + 1], bits);
    };
    switch (o >> 2) {
    case 0: from(Int<0>()); break;
    case 1: from(Int<1>()); break;
    case 2: from(Int<2>()); break;
    default: from(Int<3>()); break;
    }
}

// How many values a row begins past a 16-byte boundary.
__device__ __forceinline__ int lead_of(const uint16_t* row) { return static_cast<int>(reinterpret_cast<uintptr_t>(row) >> 1) & 7; }

// Eight values from `i` on of a row of d, zeros outside it (i may be down to -7): 16-byte
// loads, two where the first value lies off a 16-byte boundary, each holding at least
// one of the row's values.  Plain loads: the memory may be written by this kernel
// later.  kVec: every row starts aligned and holds a multiple of eight values, as i is.
template <bool kVec>
__device__ __forceinline__ void load8(const uint16_t* row, int64_t i, int64_t d, uint32_t* w)
{
    w[0] = w[1] = w[2] = w[3] = 0u;
    if (i >= d) return;
    if constexpr (kVec) {
        const uint4 v = *reinterpret_cast<const uint4*>(row + i);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else {
        const int lo = i < 0 ? static_cast<int>(-i) : 0, hi = static_cast<int>(min(static_cast<int64_t>(8), d - i));
        if (lo >= hi) return;
        const uintptr_t at = reinterpret_cast<uintptr_t>(row + i);
        const int o = static_cast<int>(at & 15u);
        const uint4* p = reinterpret_cast<const uint4*>(at - o);
        if (o == 0 && hi - lo == 8) {
            const uint4 v = *p;
            w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
            return;
        }
        uint32_t t[8] = {};
        if (2 * lo + o < 16) {
            const uint4 a = p[0];
            t[0] = a.x, t[1] = a.y, t[2] = a.z, t[3] = a.w;
        }
        if (2 * hi + o > 16) {
            const uint4 b = p[1];
            t[4] = b.x, t[5] = b.y, t[6] = b.z, t[7] = b.w;
        }
        take16(t, o, w);
        if (hi - lo < 8) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const uint32_t a = 2 * c >= lo && 2 * c < hi ? 0xFFFFu : 0u, b = 2 * c + 1 >= lo && 2 * c + 1 < hi ? 0xFFFF0000u : 0u;
                w[c] &= a | b;
            }
        }
    }
}

// Values lo to hi - 1 of eight, one by one.
__device__ __forceinline__ void store_some(uint16_t* at, const uint32_t* w, int lo, int hi)
{
#pragma unroll
    for (int c = 0; c < 8; ++c)
        if (c >= lo && c < hi) at[c] = static_cast<uint16_t>(c & 1 ? w[c >> 1] >> 16 : w[c >> 1]);
}

// Eight values from `i` on to a row of d, those inside it; row + i lies on a 16-byte
// boundary.
template <bool kVec>
__device__ __forceinline__ void store8(uint16_t* row, int64_t i, int64_t d, const uint32_t* w)
{
    if (i >= d) return;
    if (kVec || (i >= 0 && i + 8 <= d))
        *reinterpret_cast<uint4*>(row + i) = make_uint4(w[0], w[1], w[2], w[3]);
    else
        store_some(row + i, w, i < 0 ? static_cast<int>(-i) : 0, static_cast<int>(min(static_cast<int64_t>(8), d - i)));
}

// Eight values from `o` on (0 to 7) of the sixteen in a and b.
__device__ __forceinline__ void take8(const uint32_t* a, const uint32_t* b, int o, uint32_t* out)
{
    const uint32_t in[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    take16(in, 2 * o, out);
}

// The two values of a word in fp32, and back with one rounding.
template <typename T>
__device__ __forceinline__ float2 widen2(uint32_t w)
{
    return make_float2(Elem<T>::to_f32(w & 0xFFFFu), Elem<T>::to_f32(w >> 16));
}

// The sum of two such pairs, rounded once.
template <typename T>
__device__ __forceinline__ uint32_t add2(uint32_t a, uint32_t b)
{
    uint32_t r;
    if constexpr (Elem<T>::kInf == 0x7C00u)
        asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else
        asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

template <typename T>
__device__ __forceinline__ uint32_t narrow2(float a, float b);
template <>
__device__ __forceinline__ uint32_t narrow2<__half>(float a, float b)
{
    return gemm_f16_dev::pack_half2(a, b);
}
template <>
__device__ __forceinline__ uint32_t narrow2<__nv_bfloat16>(float a, float b)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

}  // namespace row_dev
