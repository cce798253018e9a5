// Activations of the products' output stages, and arithmetic on two fp32 values
// an instruction.
#pragma once

#include <cstdint>

#include "ptx.cuh"

namespace mxf4_dev {

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float rcp(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The activations without a branch, so that a thread's 32 values overlap, and of
// few instructions: with erfcf and the full division, whose rare cases branch, a
// SiLU took 220 cycles of a warp and the epilogue 9/10 of a product with K = 1000.
//
// Phi(x) for x < 0 is erfc(z) / 2 with z = -x / sqrt 2, and erfc(z) exp(z^2) is
// smooth and falls like 1 / z: t P(t) with t = 1 / (1 + z / 3) and P of degree 7,
// least relative error over 0 <= z <= 9 (fitted to the function's values in 64
// bits; gelu_factor gives half of P's), is within 1.3e-7 of it.  With the
// rounding of z^2 and the approximate exponential the whole is within 2^-18 of x
// Phi(x) wherever that is not zero in fp16.
__device__ constexpr float gelu_factor(int i)
{
    constexpr float f[8] = {0.0940747783f, 0.0931263119f, 0.0966875404f, 0.0410582423f,
                            0.168501928f,  -0.131988719f, 0.200961143f,  -0.0624212809f};
    return f[i];
}

__device__ __forceinline__ float act_f32(int act, float x)
{
    switch (act) {
    case 1: return x < 0.f ? 0.f : x;
    case 2: return x * rcp(1.f + ex2(-1.44269504f * x));
    case 3: {
        const float t = rcp(fmaf(fabsf(x), 0.70710678f / 3.f, 1.f));
        float q = gelu_factor(7);
#pragma unroll
        for (int i = 6; i >= 0; --i) q = fmaf(q, t, gelu_factor(i));
        const float h = q * t * ex2(x * x * (-0.5f * 1.44269504f));
        return x * (x < 0.f ? h : 1.f - h);
    }
    default: return x;
    }
}

// Two fp32 values an instruction.
__device__ __forceinline__ uint64_t pack2(float a, float b)
{
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
    return v;
}

__device__ __forceinline__ void unpack2(uint64_t v, float* a, float* b)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(*a), "=f"(*b) : "l"(v));
}

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t v;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(a), "l"(b), "l"(c));
    return v;
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t v;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
    return v;
}

// act_f32's GELU of two values.
__device__ __forceinline__ void gelu2(float* x0, float* x1)
{
    const uint64_t x = pack2(*x0, *x1), one = pack2(1.f, 1.f);
    auto both = [](float c) { return pack2(c, c); };
    float a, b;
    unpack2(fma2(pack2(fabsf(*x0), fabsf(*x1)), both(0.70710678f / 3.f), one), &a, &b);
    const uint64_t t = pack2(rcp(a), rcp(b));
    uint64_t q = both(gelu_factor(7));
#pragma unroll
    for (int i = 6; i >= 0; --i) q = fma2(q, t, both(gelu_factor(i)));
    unpack2(mul2(mul2(x, x), both(-0.5f * 1.44269504f)), &a, &b);
    const uint64_t h = mul2(mul2(q, t), pack2(ex2(a), ex2(b))), r = fma2(h, both(-1.f), one);
    float h0, h1, r0, r1;
    unpack2(h, &h0, &h1);
    unpack2(r, &r0, &r1);
    unpack2(mul2(x, pack2(*x0 < 0.f ? h0 : r0, *x1 < 0.f ? h1 : r1)), x0, x1);
}

// act of kN values, an even number; one choice for all of them.
template <int kN = 32>
__device__ __forceinline__ void act_all(int act, float* v)
{
    if (act == 1) {
#pragma unroll
        for (int c = 0; c < kN; ++c) v[c] = act_f32(1, v[c]);
    } else if (act == 2) {
#pragma unroll
        for (int c = 0; c < kN; ++c) v[c] = act_f32(2, v[c]);
    } else if (act == 3) {
#pragma unroll
        for (int c = 0; c < kN; c += 2) gelu2(&v[c], &v[c + 1]);
    }
}

}  // namespace mxf4_dev
