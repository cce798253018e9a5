// Tokens in the order of their experts and back: the order itself, rows copied into it,
// the experts' outputs added up by token, and that sum's gradient.  Bound by HBM, but
// for the order, whose few values are bound by latency.
//
// A choice is t * top + j; its place is its rank among all choices by expert, then by
// its own number.  Choices of no expert (an id outside 0 .. experts - 1) come last and
// have no place.
#pragma once

#include "fp8_format.cuh"
#include "rows.cuh"

namespace route_dev {

using namespace gemm_f16_dev;

constexpr int kSortThreads = 1024, kMaxExperts = 512, kMaxTop = 32;

struct SortParams {
    const int32_t* ids;
    int32_t* rows;         // place of each choice, -1: none
    int32_t* order;        // choice at each place, -1 past the last group
    int32_t* group_rows;
    int32_t* counts;       // of each part of the choices: [parts][experts + 1]
    int64_t n;             // choices
    int64_t part;          // of them a block, a multiple of 1024
    int32_t experts, parts;
};

__device__ __forceinline__ int bucket_of(const SortParams& p, int64_t i)
{
    const int e = i < p.n ? p.ids[i] : -1;
    return e >= 0 && e < p.experts ? e : p.experts;
}

// How many choices of each expert a part holds.
__global__ void __launch_bounds__(kSortThreads) sort_count(const SortParams p)
{
    __shared__ int count[kMaxExperts + 1];
    for (int e = threadIdx.x; e <= p.experts; e += kSortThreads) count[e] = 0;
    griddep_wait();
    griddep_launch_dependents();
    __syncthreads();
    const int64_t lo = static_cast<int64_t>(blockIdx.x) * p.part, hi = min(p.n, lo + p.part);
    for (int64_t i = lo + threadIdx.x; i < hi; i += kSortThreads) atomicAdd(&count[bucket_of(p, i)], 1);
    __syncthreads();
    for (int e = threadIdx.x; e <= p.experts; e += kSortThreads)
        p.counts[static_cast<int64_t>(blockIdx.x) * (p.experts + 1) + e] = count[e];
}

// Both kernels are latency: 131072 choices of 64 experts 3.5 + 8.6 us, 1024 by one block 6.
//
// The places.  Every block adds up the counts of all parts and of those before its own
// (at most 152 of them), then goes through its choices 1024 at a time: a warp finds the
// lanes of the same expert, and the warps' counts are added up in order.  One part
// (1024 choices at most) is counted here.
__global__ void __launch_bounds__(kSortThreads) sort_place(const SortParams p)
{
    constexpr int kWarps = kSortThreads / 32;
    __shared__ int total[kMaxExperts + 1], next[kMaxExperts + 1];   // choices of an expert; its next place
    __shared__ uint16_t count[kWarps][kMaxExperts + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, buckets = p.experts + 1;
    for (int e = threadIdx.x; e < buckets; e += kSortThreads) total[e] = next[e] = 0;
    for (int e = lane; e < buckets; e += 32) count[warp][e] = 0;
    griddep_wait();
    griddep_launch_dependents();
    __syncthreads();
    if (p.parts > 1) {
        int width = 32;   // threads that take neighbouring experts
        while (width < buckets) width *= 2;
        const int e = threadIdx.x & (width - 1), lots = kSortThreads / width;
        if (e < buckets) {
            int all = 0, before = 0;
#pragma unroll 16
            for (int c = threadIdx.x / width; c < p.parts; c += lots) {
                const int n = p.counts[static_cast<int64_t>(c) * buckets + e];
                all += n;
                before += c < static_cast<int>(blockIdx.x) ? n : 0;
            }
            atomicAdd(&total[e], all);
            atomicAdd(&next[e], before);
        }
    } else {
        for (int64_t i = threadIdx.x; i < p.n; i += kSortThreads) atomicAdd(&total[bucket_of(p, i)], 1);
    }
    __syncthreads();
    if (warp == 0) {   // the groups' first places
        int at = 0;
        for (int e = lane; e - lane < buckets; e += 32) {
            const int n = e < buckets ? total[e] : 0;
            int sum = n;
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const int up = __shfl_up_sync(~0u, sum, d);
                if (lane >= d) sum += up;
            }
            if (e < buckets) next[e] += at + sum - n;
            at += __shfl_sync(~0u, sum, 31);
        }
    }
    if (blockIdx.x == 0)
        for (int e = threadIdx.x; e < p.experts; e += kSortThreads) p.group_rows[e] = total[e];
    __syncthreads();
    const int64_t lo = static_cast<int64_t>(blockIdx.x) * p.part, hi = min(p.n, lo + p.part);
    for (int64_t base = lo; base < hi; base += kSortThreads) {
        const int64_t i = base + threadIdx.x;
        const bool in = i < hi;
        const int e = in ? bucket_of(p, i) : -1;
        const uint32_t same = __match_any_sync(~0u, e);
        const int rank = __popc(same & ((1u << lane) - 1));
        if (in && rank == 0) count[warp][e] = static_cast<uint16_t>(__popc(same));
        __syncthreads();
        for (int b = threadIdx.x; b < buckets; b += kSortThreads) {
            int at = 0;   // of this expert, in the warps before
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const int n = count[w][b];
                count[w][b] = static_cast<uint16_t>(at);
                at += n;
            }
            total[b] = at;
        }
        __syncthreads();
        if (in) {
            const int place = next[e] + count[warp][e] + rank;
            p.rows[i] = e < p.experts ? place : -1;
            p.order[place] = e < p.experts ? static_cast<int>(i) : -1;
        }
        __syncthreads();
        if (base + kSortThreads >= hi) break;   // (of the whole block)
        for (int b = threadIdx.x; b < buckets; b += kSortThreads) next[b] += total[b];
        for (int b = lane; b < buckets; b += 32) count[warp][b] = 0;
        __syncthreads();
    }
}

// ------------------------------------------------------------------ rows
struct RowParams {
    const uint16_t* x;       // gather: tokens; combine: places; gradient: dy, tokens
    const uint16_t* y;       // gradient: places
    uint16_t* out;           // gather and gradient: places; combine: tokens
    const int32_t* rows;
    const float* weights;    // null: ones
    float* dweights;
    int64_t sx, sy, so;      // row strides in elements
    int64_t tokens, d, places;
    int32_t top, chunks;     // chunks: blocks along a row
};

// Blocks of 128 threads, so that an SM always has some with their loads under way (256:
// combining 16384 tokens of 8 choices of 7168 values took 388 us, this 309).
constexpr int kRowThreads = 128, kChunk = kRowThreads * 8;   // values of a row a block takes at a time

// (a place outside the rows, which no order of this library holds, is taken as none)
__device__ __forceinline__ int64_t place_of(const RowParams& p, int64_t t, int j)
{
    const int64_t r = p.rows[t * p.top + j];
    return r >= 0 && r < p.places ? r : -1;
}

// A token's row is read once and written to each of its places: the other way round, by
// place, the rows would be read top times from a matrix that L2 does not hold.  Where
// rows start anywhere a thread takes the values of 16 aligned bytes of each place's row.
// 16384 tokens of 8 choices, 7168 values: 312 to 318 us (6.7 TB/s), 2049 values 159 us (3.8).
template <bool kVec>
__global__ void __launch_bounds__(kRowThreads) gather_rows(const RowParams p)
{
    const int64_t t = blockIdx.x / p.chunks, i = (blockIdx.x - t * p.chunks) * kChunk + threadIdx.x * 8;
    griddep_wait();
    griddep_launch_dependents();
    uint32_t w[4];
    if (kVec) row_dev::load8<true>(p.x + t * p.sx, i, p.d, w);
#pragma unroll 8
    for (int j = 0; j < p.top; ++j) {
        const int64_t r = place_of(p, t, j);
        if (r < 0) continue;
        uint16_t* out = p.out + r * p.so;
        const int o = kVec ? 0 : row_dev::lead_of(out);
        if (!kVec) row_dev::load8<false>(p.x + t * p.sx, i - o, p.d, w);
        row_dev::store8<kVec>(out, i - o, p.d, w);
    }
}

// The sum is in the order of the choices, in fp32, rounded once.  kAtOnce: choices whose
// rows are under way together, the more blocks an SM the fewer they are (16384 tokens of 2
// choices of 4097 values: 94 us, 187 with room for eight).
//
// 16384 tokens of 8 choices, 7168 values: 309 us (6.8 TB/s); 2049 values, rows that start
// anywhere, 238 us (2.5), by the second load and the shift of every 16 bytes.
template <typename T, bool kVec, int kAtOnce>
__global__ void __launch_bounds__(kRowThreads, kAtOnce == 8 ? 8 : kAtOnce == 4 ? 10 : kVec ? 12 : 14) combine_rows(const RowParams p)
{
    const int64_t t = blockIdx.x / p.chunks;
    uint16_t* out = p.out + t * p.so;
    const int64_t i = (blockIdx.x - t * p.chunks) * kChunk + threadIdx.x * 8 - (kVec ? 0 : row_dev::lead_of(out));
    griddep_wait();
    griddep_launch_dependents();
    float s[8] = {};
    for (int j0 = 0; j0 < p.top; j0 += kAtOnce) {
        uint32_t v[kAtOnce][4];
        float f[kAtOnce];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            const int64_t r = j0 + j < p.top ? place_of(p, t, j0 + j) : -1;
            f[j] = r < 0 ? 0.f : p.weights ? p.weights[t * p.top + j0 + j] : 1.f;
            row_dev::load8<kVec>(p.x + r * p.sx, i, r < 0 ? -8 : p.d, v[j]);
        }
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float2 a = row_dev::widen2<T>(v[j][c]);
                s[2 * c] = fmaf(f[j], a.x, s[2 * c]);
                s[2 * c + 1] = fmaf(f[j], a.y, s[2 * c + 1]);
            }
        }
    }
    uint32_t o[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) o[c] = row_dev::narrow2<T>(s[2 * c], s[2 * c + 1]);
    row_dev::store8<kVec>(out, i, p.d, o);
}

// out[place(t, j)] = w[t, j] dy[t], dweights[t, j] = dy[t] . y[place(t, j)]; a choice
// without a place has a weight's gradient of zero.  A block a token, so that the dot
// products are added up in one order.  16384 tokens of 8 choices, 7168 values: 579 us (6.9
// TB/s); 2049 values 341 us (3.4).
template <typename T, bool kVec, int kAtOnce>
__global__ void __launch_bounds__(kRowThreads, kAtOnce == 8 ? 5 : kAtOnce == 4 ? 7 : 10) combine_grad_rows(const RowParams p)
{
    __shared__ float part[kRowThreads / 32][kAtOnce];
    const int64_t t = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint16_t* dout = p.x + t * p.sx;
    griddep_wait();
    griddep_launch_dependents();
    for (int j0 = 0; j0 < p.top; j0 += kAtOnce) {
        float dot[kAtOnce] = {}, f[kAtOnce];
        int64_t at[kAtOnce];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            at[j] = j0 + j < p.top ? place_of(p, t, j0 + j) : -1;
            f[j] = at[j] < 0 ? 0.f : p.weights[t * p.top + j0 + j];
        }
        for (int64_t i = threadIdx.x * 8; i < p.d + (kVec ? 0 : 7); i += kChunk) {
            uint32_t g[4], v[kAtOnce][4];
            if (kVec) row_dev::load8<true>(dout, i, p.d, g);
            // rows that start anywhere: the values of 16 aligned bytes of dy's row
            auto lead = [&](int j) { return kVec || at[j] < 0 ? 0 : row_dev::lead_of(p.out + at[j] * p.so); };
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j)
                row_dev::load8<kVec>(p.y + at[j] * p.sy, i - lead(j), at[j] < 0 ? -8 : p.d, v[j]);
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
                if (at[j] < 0) continue;
                if (!kVec) row_dev::load8<false>(dout, i - lead(j), p.d, g);
                uint32_t o[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const float2 a = row_dev::widen2<T>(g[c]), b = row_dev::widen2<T>(v[j][c]);
                    dot[j] = fmaf(a.x, b.x, dot[j]);
                    dot[j] = fmaf(a.y, b.y, dot[j]);
                    o[c] = row_dev::narrow2<T>(f[j] * a.x, f[j] * a.y);
                }
                row_dev::store8<kVec>(p.out + at[j] * p.so, i - lead(j), p.d, o);
            }
        }
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
#pragma unroll
            for (int k = 16; k; k /= 2) dot[j] += __shfl_xor_sync(~0u, dot[j], k);
            if (lane == 0) part[warp][j] = dot[j];
        }
        __syncthreads();
        if (threadIdx.x < kAtOnce && j0 + static_cast<int>(threadIdx.x) < p.top) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < kRowThreads / 32; ++w) s += part[w][threadIdx.x];
            p.dweights[t * p.top + j0 + threadIdx.x] = s;
        }
        __syncthreads();
    }
}

// Rows held in 8 bits: the codes 16 bytes a thread, the scales a word of four blocks.  Bound
// by HBM: 16384 tokens of 8 choices, 7168 values 166 us (6.4 TB/s), 2048 values 51 (6.0), 4096
// tokens of 7168 values 44 (6.0); 16 tokens 2 us.
struct Fp8RowParams {
    const uint8_t *codes, *scales;
    uint8_t *out_codes, *out_scales;
    const int32_t* rows;
    int64_t tokens, places, pitch, kt;
    int32_t top, chunks;
};

__global__ void __launch_bounds__(kRowThreads) gather_fp8(const Fp8RowParams p)
{
    const int64_t t = blockIdx.x / p.chunks, c = (blockIdx.x - t * p.chunks) * kRowThreads + threadIdx.x;
    griddep_wait();
    griddep_launch_dependents();
    if (t == p.tokens) {   // the last block: padding rows of the last scale tile
        const int64_t end = (p.places + 127) / 128 * 128;
        for (int64_t i = threadIdx.x; i < (end - p.places) * p.kt; i += kRowThreads)
            *reinterpret_cast<uint32_t*>(p.out_scales + fp8_dev::scale_at(p.places + i / p.kt, 4 * (i % p.kt), p.kt)) = 0u;
        return;
    }
    const bool code = c * 16 < p.pitch, scale = c < p.kt;
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    uint32_t s = 0u;
    if (code) v = ld_nc_v4(p.codes + t * p.pitch + c * 16);
    if (scale) s = ld_nc_u32(p.scales + fp8_dev::scale_at(t, 4 * c, p.kt));
#pragma unroll 8
    for (int j = 0; j < p.top; ++j) {
        const int64_t r = p.rows[t * p.top + j];
        if (r < 0 || r >= p.places) continue;
        if (code) *reinterpret_cast<uint4*>(p.out_codes + r * p.pitch + c * 16) = v;
        if (scale) *reinterpret_cast<uint32_t*>(p.out_scales + fp8_dev::scale_at(r, 4 * c, p.kt)) = s;
    }
}

}  // namespace route_dev
