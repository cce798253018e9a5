// Host side of the norm (rms_norm.h): argument checks, the choice of form, the launch.
#include <cmath>
#include <cstdint>

#include "gemm_fp8.h"
#include "host.h"
#include "rms_norm.cuh"
#include "rms_norm.h"

using namespace gemm_f16_host;

namespace {

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

template <typename T, int kMost, int kVecs>
gemm_f16_status launch(const norm_dev::Params& p, bool vec, int threads, cudaStream_t stream)
{
    const int64_t blocks = kMost == 256 ? cdiv(p.rows, kMost / 32) : p.rows;
    if (blocks > INT32_MAX) return GEMM_F16_ERR_INVALID_VALUE;
    return launch_kernel(vec ? norm_dev::rms_norm<T, kMost, kVecs, true> : norm_dev::rms_norm<T, kMost, kVecs, false>,
                         dim3(static_cast<unsigned>(blocks)), static_cast<unsigned>(threads), 0, 1, stream, p);
}

template <typename T>
gemm_f16_status choose(const norm_dev::Params& p, bool vec, int sms, cudaStream_t stream)
{
    const int64_t d = p.d + (vec ? 0 : 7);   // (a row that starts up to 7 values past a boundary)
    if (d <= 256) return launch<T, 256, 1>(p, vec, 256, stream);
    if (d <= 512) return launch<T, 256, 2>(p, vec, 256, stream);
    if (d <= 1024) return launch<T, 256, 4>(p, vec, 256, stream);
    auto threads = [&](int vecs) { return static_cast<int>(cdiv(d, 256 * vecs) * 32); };
    // few rows: as many threads as a row has work for
    if (p.rows <= sms && threads(1) <= 1024) return launch<T, 1024, 1>(p, vec, threads(1), stream);
    // otherwise 2 to 4 times 8 values a thread, whichever leaves the fewest without
    int vecs = 4;
    for (int v = 3; v >= 2; --v)
        if (v * threads(v) < vecs * threads(vecs)) vecs = v;
    if (threads(4) > 288) return launch<T, 832, 5>(p, vec, threads(5), stream);
    return vecs == 4   ? launch<T, 288, 4>(p, vec, threads(4), stream)
           : vecs == 3 ? launch<T, 384, 3>(p, vec, threads(3), stream)
                       : launch<T, 576, 2>(p, vec, threads(2), stream);
}

}  // namespace

extern "C" gemm_f16_status rms_norm(const void* x, int dtype, int64_t stride_x, const void* residual,
                                    int64_t stride_residual, const void* weight, float eps, void* sum,
                                    int64_t stride_sum, void* y, int64_t stride_y, void* codes, void* scales,
                                    int64_t rows, int64_t d, cudaStream_t stream)
{
    if (dtype < FP8_F16 || dtype > FP8_BF16 || rows < 0 || rows > GEMM_F16_MAX_DIM || d < 1 || d > RMS_NORM_MAX_DIM ||
        !std::isfinite(eps) || eps < 0.f)
        return GEMM_F16_ERR_INVALID_VALUE;
    if (rows == 0) return GEMM_F16_OK;
    const bool q = y == nullptr;
    if (!x || !weight || !residual != !sum || (q ? !codes || !scales : codes || scales)) return GEMM_F16_ERR_INVALID_VALUE;
    if (!aligned(x, 2) || !aligned(residual, 2) || !aligned(weight, 2) || !aligned(sum, 2) || !aligned(y, 2) ||
        !aligned(codes, 16) || !aligned(scales, 16))
        return GEMM_F16_ERR_INVALID_VALUE;
    struct Range {
        const void* p;
        int64_t stride, bytes;
    } in[] = {{x, stride_x, 0}, {residual, stride_residual, 0}, {sum, stride_sum, 0}, {y, stride_y, 0}};
    for (Range& r : in) {
        if (!r.p) continue;
        if (r.stride < d || !view_extent(rows, d, r.stride, 1, &r.bytes) || __builtin_mul_overflow(r.bytes, 2, &r.bytes))
            return GEMM_F16_ERR_INVALID_VALUE;
    }
    int64_t code_bytes = 0, scale_bytes = 0;
    if (q) {
        const gemm_f16_status st = fp8_sizes(rows, d, 1, &code_bytes, &scale_bytes);
        if (st != GEMM_F16_OK) return st;
    }
    const Range out[] = {{y, 0, in[3].bytes}, {codes, 0, code_bytes}, {scales, 0, scale_bytes}};
    auto clash = [](const Range& a, const Range& b) { return a.p && b.p && overlaps(a.p, a.bytes, b.p, b.bytes); };
    const Range w{weight, 0, 2 * d};
    for (const Range& o : out)
        if (clash(o, in[0]) || clash(o, in[1]) || clash(o, in[2]) || clash(o, w)) return GEMM_F16_ERR_ALIAS;
    if (clash(out[1], out[2]) || clash(in[2], w)) return GEMM_F16_ERR_ALIAS;
    for (int i = 0; i < 2; ++i)   // in place is fine: a thread reads its values before it writes them
        if (clash(in[2], in[i]) && !(in[2].p == in[i].p && in[2].stride == in[i].stride)) return GEMM_F16_ERR_ALIAS;
    Device dev;
    const gemm_f16_status st = current_device(&dev);
    if (st != GEMM_F16_OK) return st;
    for (const Range& r : in)
        if (r.p && !device_range_ok(r.p, r.bytes)) return GEMM_F16_ERR_INVALID_VALUE;
    if (!device_range_ok(weight, w.bytes) || (q && (!device_range_ok(codes, code_bytes) || !device_range_ok(scales, scale_bytes))))
        return GEMM_F16_ERR_INVALID_VALUE;
    norm_dev::Params p = {};
    p.x = static_cast<const uint16_t*>(x);
    p.residual = static_cast<const uint16_t*>(residual);
    p.weight = static_cast<const uint16_t*>(weight);
    p.sum = static_cast<uint16_t*>(sum);
    p.y = static_cast<uint16_t*>(y);
    p.codes = static_cast<uint8_t*>(codes);
    p.scales = static_cast<uint8_t*>(scales);
    p.sx = stride_x, p.sr = stride_residual, p.ss = stride_sum, p.sy = stride_y;
    p.rows = rows, p.d = d, p.pitch = cdiv(d, 128) * 128, p.kt = cdiv(d, 512), p.row_tiles = cdiv(rows, 128);
    p.eps = eps;
    bool vec = d % 8 == 0 && aligned(weight, 16);
    for (const Range& r : in)
        if (r.p) vec = vec && aligned(r.p, 16) && r.stride % 8 == 0;
    return dtype == FP8_F16 ? choose<__half>(p, vec, dev.sms, stream) : choose<__nv_bfloat16>(p, vec, dev.sms, stream);
}
