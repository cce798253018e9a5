// Host side of the expert order (moe_route.h): argument checks and launches.
#include <algorithm>
#include <cstdint>

#include "gemm_fp8.h"
#include "host.h"
#include "moe_route.cuh"
#include "moe_route.h"

using namespace gemm_f16_host;

static_assert(MOE_ROUTE_MAX_EXPERTS == route_dev::kMaxExperts && MOE_ROUTE_MAX_TOP_K == route_dev::kMaxTop,
              "the header and the kernels agree on the limits");

namespace {

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// Parts of the choices that moe_sort counts by themselves: one block each, at most 152,
// so that every block can add up all counts.  (A block for each SM of a GB300; a constant,
// because the workspace's size hangs on it and is asked for where no device is.)  One block
// alone takes 1024 choices at once; 4096 took it 18 us, two kernels 10.
constexpr int64_t kFewChoices = 1024, kMaxParts = 152;

bool sort_parts(int64_t tokens, int64_t top, int64_t experts, int64_t* part, int64_t* parts)
{
    if (tokens < 0 || tokens > GEMM_F16_MAX_DIM || top < 1 || top > MOE_ROUTE_MAX_TOP_K || experts < 1 ||
        experts > MOE_ROUTE_MAX_EXPERTS || tokens * top > GEMM_F16_MAX_DIM)
        return false;
    const int64_t n = tokens * top;
    *part = n <= kFewChoices ? kFewChoices : cdiv(cdiv(n, kMaxParts), 1024) * 1024;
    *parts = std::max<int64_t>(1, cdiv(n, *part));
    return true;
}

size_t sort_bytes(int64_t parts, int64_t experts) { return parts > 1 ? static_cast<size_t>(parts * (experts + 1) * 4) : 0; }

struct Range {
    const void* p;
    int64_t bytes;
};

bool clash(const Range& a, const Range& b) { return a.p && b.p && overlaps(a.p, a.bytes, b.p, b.bytes); }

// Outputs overlap no input and not each other; everything is memory of the device.
template <size_t kIn, size_t kOut>
gemm_f16_status check(const Range (&in)[kIn], const Range (&out)[kOut], Device* dev)
{
    for (size_t o = 0; o < kOut; ++o) {
        for (const Range& r : in)
            if (clash(out[o], r)) return GEMM_F16_ERR_ALIAS;
        for (size_t q = 0; q < o; ++q)
            if (clash(out[o], out[q])) return GEMM_F16_ERR_ALIAS;
    }
    const gemm_f16_status st = current_device(dev);
    if (st != GEMM_F16_OK) return st;
    for (const Range& r : in)
        if (r.p && !device_range_ok(r.p, r.bytes)) return GEMM_F16_ERR_INVALID_VALUE;
    for (const Range& r : out)
        if (r.p && !device_range_ok(r.p, r.bytes)) return GEMM_F16_ERR_INVALID_VALUE;
    return GEMM_F16_OK;
}

// The bytes of a matrix of 16-bit rows; false unless its address and strides are fine.
bool rows_of(const void* p, int64_t rows, int64_t d, int64_t stride, Range* r)
{
    r->p = p;
    return p && aligned(p, 2) && stride >= d && view_extent(rows, d, stride, 1, &r->bytes) &&
           !__builtin_mul_overflow(r->bytes, 2, &r->bytes);
}

bool sizes_ok(int dtype, const int32_t* rows, int64_t tokens, int64_t top, int64_t d)
{
    return dtype >= FP8_F16 && dtype <= FP8_BF16 && tokens >= 0 && tokens <= GEMM_F16_MAX_DIM && top >= 1 &&
           top <= MOE_ROUTE_MAX_TOP_K && tokens * top <= GEMM_F16_MAX_DIM && d >= 1 && d <= GEMM_F16_MAX_DIM &&
           (tokens == 0 || (rows && aligned(rows, 4)));
}

bool takes_vectors(const void* p, int64_t stride) { return !p || (aligned(p, 16) && stride % 8 == 0); }

// Blocks along a row; one that starts up to 7 values past a 16-byte boundary reaches
// that much further.
int32_t chunks_of(int64_t d, bool vec) { return static_cast<int32_t>(cdiv(d + (vec ? 0 : 7), route_dev::kChunk)); }

gemm_f16_status launch_rows(void (*kernel)(const route_dev::RowParams), const route_dev::RowParams& p, int64_t blocks,
                            cudaStream_t stream)
{
    if (blocks > INT32_MAX) return GEMM_F16_ERR_INVALID_VALUE;
    return launch_kernel(kernel, dim3(static_cast<unsigned>(blocks)), route_dev::kRowThreads, 0, 1, stream, p);
}

}  // namespace

extern "C" {

gemm_f16_status moe_sort_workspace_size(int64_t tokens, int64_t top_k, int64_t experts, size_t* bytes)
{
    int64_t part, parts;
    if (!bytes || !sort_parts(tokens, top_k, experts, &part, &parts)) return GEMM_F16_ERR_INVALID_VALUE;
    *bytes = sort_bytes(parts, experts);
    return GEMM_F16_OK;
}

gemm_f16_status moe_sort(const int32_t* ids, int64_t tokens, int64_t top_k, int64_t experts, int32_t* rows,
                         int32_t* order, int32_t* group_rows, void* workspace, size_t workspace_bytes,
                         cudaStream_t stream)
{
    int64_t part, parts;
    if (!sort_parts(tokens, top_k, experts, &part, &parts) || !group_rows || (tokens && (!ids || !rows || !order)))
        return GEMM_F16_ERR_INVALID_VALUE;
    if (!aligned(ids, 4) || !aligned(rows, 4) || !aligned(order, 4) || !aligned(group_rows, 4)) return GEMM_F16_ERR_INVALID_VALUE;
    const size_t need = sort_bytes(parts, experts);
    if (need && (!workspace || workspace_bytes < need || !aligned(workspace, 256))) return GEMM_F16_ERR_OUT_OF_MEMORY;
    const int64_t n = tokens * top_k;
    const Range in[] = {{n ? ids : nullptr, 4 * n}};
    const Range out[] = {{n ? rows : nullptr, 4 * n}, {n ? order : nullptr, 4 * n}, {group_rows, 4 * experts},
                         {need ? workspace : nullptr, static_cast<int64_t>(need)}};
    Device dev;
    gemm_f16_status st = check(in, out, &dev);
    if (st != GEMM_F16_OK) return st;
    route_dev::SortParams p = {};
    p.ids = ids, p.rows = rows, p.order = order, p.group_rows = group_rows, p.counts = static_cast<int32_t*>(workspace);
    p.n = n, p.part = part, p.experts = static_cast<int32_t>(experts), p.parts = static_cast<int32_t>(parts);
    const dim3 grid(static_cast<unsigned>(parts));
    if (parts > 1) {
        st = launch_kernel(route_dev::sort_count, grid, route_dev::kSortThreads, 0, 1, stream, p);
        if (st != GEMM_F16_OK) return st;
    }
    return launch_kernel(route_dev::sort_place, grid, route_dev::kSortThreads, 0, 1, stream, p);
}

gemm_f16_status moe_gather(const void* x, int dtype, int64_t stride_x, const int32_t* rows, int64_t tokens,
                           int64_t top_k, int64_t d, void* out, int64_t stride_out, cudaStream_t stream)
{
    if (!sizes_ok(dtype, rows, tokens, top_k, d)) return GEMM_F16_ERR_INVALID_VALUE;
    if (tokens == 0) return GEMM_F16_OK;
    const int64_t n = tokens * top_k;
    Range rx, ro;
    if (!rows_of(x, tokens, d, stride_x, &rx) || !rows_of(out, n, d, stride_out, &ro)) return GEMM_F16_ERR_INVALID_VALUE;
    const Range in[] = {rx, {rows, 4 * n}}, outs[] = {ro};
    Device dev;
    const gemm_f16_status st = check(in, outs, &dev);
    if (st != GEMM_F16_OK) return st;
    route_dev::RowParams p = {};
    p.x = static_cast<const uint16_t*>(x), p.out = static_cast<uint16_t*>(out), p.rows = rows;
    p.sx = stride_x, p.so = stride_out, p.tokens = tokens, p.d = d, p.places = n;
    const bool vec = d % 8 == 0 && takes_vectors(x, stride_x) && takes_vectors(out, stride_out);
    p.top = static_cast<int32_t>(top_k), p.chunks = chunks_of(d, vec);
    return launch_rows(vec ? route_dev::gather_rows<true> : route_dev::gather_rows<false>, p, tokens * p.chunks, stream);
}

gemm_f16_status moe_gather_fp8(const void* codes, const void* scales, const int32_t* rows, int64_t tokens,
                               int64_t top_k, int64_t k, void* out_codes, void* out_scales, cudaStream_t stream)
{
    if (!sizes_ok(FP8_F16, rows, tokens, top_k, k)) return GEMM_F16_ERR_INVALID_VALUE;
    if (tokens == 0) return GEMM_F16_OK;
    const int64_t n = tokens * top_k;
    if (!codes || !scales || !out_codes || !out_scales || !aligned(codes, 16) || !aligned(scales, 16) ||
        !aligned(out_codes, 16) || !aligned(out_scales, 16))
        return GEMM_F16_ERR_INVALID_VALUE;
    int64_t cb, sb, ocb, osb;
    gemm_f16_status st = fp8_sizes(tokens, k, 1, &cb, &sb);
    if (st == GEMM_F16_OK) st = fp8_sizes(n, k, 1, &ocb, &osb);
    if (st != GEMM_F16_OK) return st;
    const Range in[] = {{codes, cb}, {scales, sb}, {rows, 4 * n}}, out[] = {{out_codes, ocb}, {out_scales, osb}};
    Device dev;
    st = check(in, out, &dev);
    if (st != GEMM_F16_OK) return st;
    route_dev::Fp8RowParams p = {};
    p.codes = static_cast<const uint8_t*>(codes), p.scales = static_cast<const uint8_t*>(scales);
    p.out_codes = static_cast<uint8_t*>(out_codes), p.out_scales = static_cast<uint8_t*>(out_scales);
    p.rows = rows, p.tokens = tokens, p.places = n, p.pitch = cdiv(k, 128) * 128, p.kt = cdiv(k, 512);
    p.top = static_cast<int32_t>(top_k), p.chunks = static_cast<int32_t>(cdiv(p.pitch, 16 * route_dev::kRowThreads));
    const int64_t blocks = tokens * p.chunks + 1;   // the last one: padding
    if (blocks > INT32_MAX) return GEMM_F16_ERR_INVALID_VALUE;
    return launch_kernel(route_dev::gather_fp8, dim3(static_cast<unsigned>(blocks)), route_dev::kRowThreads, 0, 1, stream, p);
}

gemm_f16_status moe_combine(const void* y, int dtype, int64_t stride_y, const int32_t* rows, const float* weights,
                            int64_t tokens, int64_t top_k, int64_t d, void* out, int64_t stride_out,
                            cudaStream_t stream)
{
    if (!sizes_ok(dtype, rows, tokens, top_k, d)) return GEMM_F16_ERR_INVALID_VALUE;
    if (tokens == 0) return GEMM_F16_OK;
    const int64_t n = tokens * top_k;
    Range ry, ro;
    if (!rows_of(y, n, d, stride_y, &ry) || !rows_of(out, tokens, d, stride_out, &ro) || !aligned(weights, 4))
        return GEMM_F16_ERR_INVALID_VALUE;
    const Range in[] = {ry, {rows, 4 * n}, {weights, 4 * n}}, outs[] = {ro};
    Device dev;
    const gemm_f16_status st = check(in, outs, &dev);
    if (st != GEMM_F16_OK) return st;
    route_dev::RowParams p = {};
    p.x = static_cast<const uint16_t*>(y), p.out = static_cast<uint16_t*>(out), p.rows = rows, p.weights = weights;
    p.sx = stride_y, p.so = stride_out, p.tokens = tokens, p.d = d, p.places = n;
    const bool vec = d % 8 == 0 && takes_vectors(y, stride_y) && takes_vectors(out, stride_out), half = dtype == FP8_F16;
    p.top = static_cast<int32_t>(top_k), p.chunks = chunks_of(d, vec);
    auto kernel = [&](auto type, auto vectors) {
        using T = decltype(type);
        constexpr bool kVec = decltype(vectors)::value;
        return top_k <= 2   ? route_dev::combine_rows<T, kVec, 2>
               : top_k <= 4 ? route_dev::combine_rows<T, kVec, 4>
                            : route_dev::combine_rows<T, kVec, 8>;
    };
    using fp8_dev::Bool;
    return launch_rows(half ? (vec ? kernel(__half(), Bool<true>()) : kernel(__half(), Bool<false>()))
                            : (vec ? kernel(__nv_bfloat16(), Bool<true>()) : kernel(__nv_bfloat16(), Bool<false>())),
                       p, tokens * p.chunks, stream);
}

gemm_f16_status moe_combine_grad(const void* dout, int dtype, int64_t stride_dout, const void* y, int64_t stride_y,
                                 const int32_t* rows, const float* weights, int64_t tokens, int64_t top_k, int64_t d,
                                 void* dy, int64_t stride_dy, float* dweights, cudaStream_t stream)
{
    if (!sizes_ok(dtype, rows, tokens, top_k, d)) return GEMM_F16_ERR_INVALID_VALUE;
    if (tokens == 0) return GEMM_F16_OK;
    const int64_t n = tokens * top_k;
    Range rg, ry, rd;
    if (!rows_of(dout, tokens, d, stride_dout, &rg) || !rows_of(y, n, d, stride_y, &ry) ||
        !rows_of(dy, n, d, stride_dy, &rd) || !weights || !dweights || !aligned(weights, 4) || !aligned(dweights, 4))
        return GEMM_F16_ERR_INVALID_VALUE;
    const Range in[] = {rg, ry, {rows, 4 * n}, {weights, 4 * n}}, out[] = {rd, {dweights, 4 * n}};
    Device dev;
    const gemm_f16_status st = check(in, out, &dev);
    if (st != GEMM_F16_OK) return st;
    route_dev::RowParams p = {};
    p.x = static_cast<const uint16_t*>(dout), p.y = static_cast<const uint16_t*>(y), p.out = static_cast<uint16_t*>(dy);
    p.rows = rows, p.weights = weights, p.dweights = dweights;
    p.sx = stride_dout, p.sy = stride_y, p.so = stride_dy, p.tokens = tokens, p.d = d, p.places = n;
    p.top = static_cast<int32_t>(top_k);
    const bool vec = d % 8 == 0 && takes_vectors(dout, stride_dout) && takes_vectors(y, stride_y) && takes_vectors(dy, stride_dy);
    const bool half = dtype == FP8_F16;
    auto kernel = [&](auto type, auto vectors) {
        using T = decltype(type);
        constexpr bool kVec = decltype(vectors)::value;   // (rows that start anywhere: two loads each)
        return top_k <= 2           ? route_dev::combine_grad_rows<T, kVec, 2>
               : top_k <= 4 || !kVec ? route_dev::combine_grad_rows<T, kVec, 4>
                                     : route_dev::combine_grad_rows<T, kVec, kVec ? 8 : 4>;
    };
    using fp8_dev::Bool;
    return launch_rows(half ? (vec ? kernel(__half(), Bool<true>()) : kernel(__half(), Bool<false>()))
                            : (vec ? kernel(__nv_bfloat16(), Bool<true>()) : kernel(__nv_bfloat16(), Bool<false>())),
                       p, tokens, stream);
}

}  // extern "C"
