// Rows of 16-bit values, eight a lane and 256 a warp: loads and stores of rows that
// start at any element.
#pragma once

#include "mxf4_format.cuh"

namespace row_dev {

using mxf4_dev::Elem;
using mxf4_dev::funnel16;

// Eight values from `i` on of a row of d (zeros past it): 16-byte loads, two where the
// row starts off a 16-byte boundary, each holding at least one of the values.  Plain
// loads: the memory may be written by this kernel later.  kVec: every row starts
// aligned and holds a multiple of eight values.
template <bool kVec>
__device__ __forceinline__ void load8(const uint16_t* row, int64_t i, int64_t d, uint32_t* w)
{
    w[0] = w[1] = w[2] = w[3] = 0u;
    if (i >= d) return;
    if constexpr (kVec) {
        const uint4 v = *reinterpret_cast<const uint4*>(row + i);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else {
        const uintptr_t at = reinterpret_cast<uintptr_t>(row + i);
        const uint32_t o = at & 15u;
        const uint4* p = reinterpret_cast<const uint4*>(at - o);
        const int n = static_cast<int>(min(static_cast<int64_t>(8), d - i));
        uint32_t t[8] = {};
        const uint4 a = p[0];
        t[0] = a.x, t[1] = a.y, t[2] = a.z, t[3] = a.w;
        if (2 * n + static_cast<int>(o) > 16) {
            const uint4 b = p[1];
            t[4] = b.x, t[5] = b.y, t[6] = b.z, t[7] = b.w;
        }
        funnel16(t, o, w);
        if (n < 8) mxf4_dev::mask_tail<__half>(w, n);
    }
}

// Values lo to hi - 1 of eight, one by one.
__device__ __forceinline__ void store_some(uint16_t* at, const uint32_t* w, int lo, int hi)
{
#pragma unroll
    for (int c = 0; c < 8; ++c)
        if (c >= lo && c < hi) at[c] = static_cast<uint16_t>(c & 1 ? w[c >> 1] >> 16 : w[c >> 1]);
}

// The inverse, by all lanes of a warp whose values follow one another.  Where the row
// starts off a boundary by o values a lane stores the 16 aligned bytes that end in its
// own values, with the last o of the lane before it; the first lane has its own 8 - o
// one by one, and the last lane its last o.
template <bool kVec>
__device__ __forceinline__ void store8(uint16_t* row, int64_t i, int64_t d, const uint32_t* w)
{
    uint16_t* at = row + i;
    if constexpr (kVec) {
        if (i < d) *reinterpret_cast<uint4*>(at) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
        const int o = static_cast<int>(reinterpret_cast<uintptr_t>(at) >> 1) & 7;
        auto left = [&](int64_t from) { return static_cast<int>(max(int64_t(0), min(int64_t(8), d - from))); };
        if (o == 0) {
            if (i + 8 <= d)
                *reinterpret_cast<uint4*>(at) = make_uint4(w[0], w[1], w[2], w[3]);
            else
                store_some(at, w, 0, left(i));
            return;
        }
        const int lane = threadIdx.x & 31;
        uint32_t in[8], out[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            in[c] = __shfl_up_sync(~0u, w[c], 1);
            in[4 + c] = w[c];
        }
        funnel16(in, 16 - 2 * o, out);
        if (lane > 0 && i - o + 8 <= d)
            *reinterpret_cast<uint4*>(at - o) = make_uint4(out[0], out[1], out[2], out[3]);
        else
            store_some(at - o, out, lane ? 0 : o, left(i - o));
        if (lane == 31) store_some(at, w, 8 - o, left(i));
    }
}

// The two values of a word in fp32, and back with one rounding.
template <typename T>
__device__ __forceinline__ float2 widen2(uint32_t w)
{
    return make_float2(Elem<T>::to_f32(w & 0xFFFFu), Elem<T>::to_f32(w >> 16));
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
