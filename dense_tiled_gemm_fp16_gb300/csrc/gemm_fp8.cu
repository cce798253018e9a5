// Host side of the 8-bit entry points (gemm_fp8.h): argument checks, the choice of
// form, tensor maps and launches.
#include <algorithm>
#include <cstdint>
#include <mutex>

#include "fp8_convert.cuh"
#include "fp8_gemm.cuh"
#include "gemm_fp8.h"
#include "host.h"

using namespace gemm_f16_host;

namespace {

constexpr int kMaxSmem = 232448;
constexpr int64_t kMaxBatch = 65535;   // batches are the third grid dimension

struct Sizes {
    int64_t pitch, kt, row_tiles, code_bytes, scale_bytes;   // bytes of the whole batch
};

bool sizes_of(int64_t rows, int64_t k, int64_t batch, Sizes* s)
{
    if (rows < 1 || k < 1 || batch < 1 || rows > GEMM_F16_MAX_DIM || k > GEMM_F16_MAX_DIM) return false;
    s->pitch = cdiv(k, 128) * 128;
    s->kt = cdiv(k, 512);
    s->row_tiles = cdiv(rows, 128);
    if (__builtin_mul_overflow(rows * s->pitch, batch, &s->code_bytes)) return false;
    return !__builtin_mul_overflow(s->row_tiles * s->kt * fp8_dev::kScaleTile, batch, &s->scale_bytes);
}

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

int64_t elem_bytes(int dtype) { return dtype == FP8_F32 ? 4 : 2; }

// Codes as {pitch bytes, rows, matrices}, boxes of 128 bytes x box_rows.
bool encode_codes(CUtensorMap* tm, const void* codes, int64_t rows, int64_t batch, int64_t pitch, uint32_t box_rows)
{
    const auto encode = tensor_map_encoder();
    if (!encode) return false;
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(pitch), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(batch)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(pitch), static_cast<cuuint64_t>(rows * pitch)};
    cuuint32_t box[3] = {128, box_rows, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return encode(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, batch ? 3 : 2, const_cast<void*>(codes), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// C, boxes of 32 rows x the columns of an epilogue's warp: 32, of a gated product 16.
bool encode_out(CUtensorMap* tm, void* C, int64_t M, int64_t N, int64_t ldc, bool gated)
{
    const auto encode = tensor_map_encoder();
    if (!encode) return false;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(M)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(2 * ldc)};
    cuuint32_t box[2] = {gated ? 16u : 32u, 32};
    cuuint32_t estr[2] = {1, 1};
    return encode(tm, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, C, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  gated ? CU_TENSOR_MAP_SWIZZLE_32B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Dynamic shared memory above 48 KB is allowed once per device and kernel.
bool allow_smem(const void* kernel, int slot, int bytes)
{
    static std::mutex mutex;
    static bool done[64][3] = {};
    int d = 0;
    if (cudaGetDevice(&d) != cudaSuccess || d < 0 || d >= 64) {
        cudaGetLastError();
        return false;
    }
    std::lock_guard<std::mutex> lk(mutex);
    if (!done[d][slot]) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) {
            cudaGetLastError();
            return false;
        }
        done[d][slot] = true;
    }
    return true;
}

template <typename T>
gemm_f16_status launch_quantize(fp8_dev::QuantParams p, int64_t batch, cudaStream_t stream)
{
    const bool rows = p.sk == 1, vec = aligned(p.x, 16) && p.sr * sizeof(T) % 16 == 0 && p.sb * sizeof(T) % 16 == 0;
    if (!rows) p.tile_rows = fp8_dev::kTileRows;
    const int64_t blocks = cdiv(p.rows, p.tile_rows) * p.kt;
    if (blocks > INT32_MAX) return GEMM_F16_ERR_INVALID_VALUE;
    const auto kernel = !rows ? fp8_dev::quantize_strided<T>
                        : vec ? fp8_dev::quantize_rows<T, true>
                              : fp8_dev::quantize_rows<T, false>;
    return launch_kernel(kernel, dim3(static_cast<unsigned>(blocks), 1, static_cast<unsigned>(batch)), fp8_dev::kConvThreads,
                         0, 1, stream, p);
}

gemm_f16_status run_quantize(const void* x, int dtype, int64_t sb, int64_t sr, int64_t sk, void* codes, void* scales,
                             int64_t rows, int64_t k, int64_t batch, const Sizes& s, int sms, cudaStream_t stream)
{
    // Rows of a block: 32 of many tiles, fewer of few, so that there are blocks for every SM.
    // A row a warp (8) against 16: 1.5 and 2.1 us at 16 x 8192 (16 tiles), 3.7 and 3.8 at
    // 1024 x 4096 (64), but 6.0 and 5.7 at 2048 x 4096 (128), 8.2 and 7.5 at 3001 x 4096 (192).
    // 16, 32, 64, 128: 14.9, 14.6, 17.1, 19.1 at 4096 x 7168 (448 tiles), 56, 54, 55, 61 at
    // 16384 x 7168, 427, 408, 407, 410 at 131072 x 7168 (all bf16).
    const int64_t tiles = s.row_tiles * s.kt * batch, tile_rows = tiles >= 2 * sms ? 32 : 2 * tiles >= sms ? 16 : 8;
    const fp8_dev::QuantParams p{x, sb, sr, sk, static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales), rows, k,
                                 s.pitch, s.kt, s.row_tiles, tile_rows};
    return dtype == FP8_F16    ? launch_quantize<__half>(p, batch, stream)
           : dtype == FP8_BF16 ? launch_quantize<__nv_bfloat16>(p, batch, stream)
                               : launch_quantize<float>(p, batch, stream);
}

template <typename T>
gemm_f16_status launch_dequantize(const fp8_dev::DequantParams& p, int64_t batch, cudaStream_t stream)
{
    const int64_t blocks = cdiv(p.rows, fp8_dev::kDequantRows) * p.col_tiles;
    if (blocks > INT32_MAX) return GEMM_F16_ERR_INVALID_VALUE;
    const dim3 grid(static_cast<unsigned>(blocks), 1, static_cast<unsigned>(batch));
    return launch_kernel(p.k % 8 == 0 && aligned(p.y, 16) ? fp8_dev::dequantize<T, true> : fp8_dev::dequantize<T, false>,
                         grid, fp8_dev::kConvThreads, 0, 1, stream, p);
}

// What the products' entry points are given, checked by check().
struct Product {
    const void *a_codes, *a_scales;            // null where `a` is quantised into `work`
    const void* a;
    int a_dtype;
    int64_t sm, sk;
    void* work;
    const void *b_codes, *b_scales, *u_codes, *u_scales;
    const void* bias;
    const int32_t* group_rows;
    int act;
    void* c;
    int dtype;
    int64_t ldc, m, n, k, groups;   // groups: 0 for the single product
};

gemm_f16_status check(const Product& q, Sizes* sa, Sizes* sb, Device* dev)
{
    const bool held = q.a == nullptr;
    if (q.groups < 0 || q.groups > GEMM_FP8_MAX_GROUPS || !sizes_of(q.m, q.k, 1, sa) ||
        !sizes_of(q.n, q.k, std::max<int64_t>(q.groups, 1), sb))
        return GEMM_F16_ERR_INVALID_VALUE;
    if (!q.b_codes || !q.b_scales || !q.c || (held && (!q.a_codes || !q.a_scales)) || (!held && !q.work) ||
        (q.groups && !q.group_rows) || !q.u_codes != !q.u_scales)
        return GEMM_F16_ERR_INVALID_VALUE;
    if (q.act < GEMM_F16_ACT_NONE || q.act > GEMM_F16_ACT_GELU || q.dtype < FP8_F16 || q.dtype > FP8_BF16 || q.ldc < q.n)
        return GEMM_F16_ERR_INVALID_VALUE;
    if (!aligned(q.b_codes, 16) || !aligned(q.b_scales, 16) || !aligned(q.u_codes, 16) || !aligned(q.u_scales, 16) ||
        !aligned(q.a_codes, 16) || !aligned(q.a_scales, 16) || !aligned(q.work, 16) || !aligned(q.a, 2) ||
        !aligned(q.c, 2) || !aligned(q.bias, 2) || !aligned(q.group_rows, 4))
        return GEMM_F16_ERR_INVALID_VALUE;
    int64_t c_bytes, a_bytes = 0, work_bytes = 0;
    if (!view_extent(q.m, q.n, q.ldc, 1, &c_bytes) || __builtin_mul_overflow(c_bytes, 2, &c_bytes))
        return GEMM_F16_ERR_INVALID_VALUE;
    if (!held) {
        if (q.a_dtype < FP8_F16 || q.a_dtype > FP8_BF16 || q.sm <= 0 || q.sk <= 0 ||
            !view_extent(q.m, q.k, q.sm, q.sk, &a_bytes) || __builtin_mul_overflow(a_bytes, 2, &a_bytes) ||
            __builtin_add_overflow(sa->code_bytes, sa->scale_bytes, &work_bytes))
            return GEMM_F16_ERR_INVALID_VALUE;
    }
    struct Range {
        const void* p;
        int64_t bytes;
    };
    const Range in[] = {{q.a_codes, sa->code_bytes}, {q.a_scales, sa->scale_bytes}, {q.a, a_bytes},
                        {q.b_codes, sb->code_bytes}, {q.b_scales, sb->scale_bytes}, {q.u_codes, sb->code_bytes},
                        {q.u_scales, sb->scale_bytes}, {q.bias, 2 * q.n}, {q.group_rows, 4 * q.groups}};
    for (const Range& r : in)
        if (r.p && (overlaps(q.c, c_bytes, r.p, r.bytes) || (!held && overlaps(q.work, work_bytes, r.p, r.bytes))))
            return GEMM_F16_ERR_ALIAS;
    if (!held && overlaps(q.c, c_bytes, q.work, work_bytes)) return GEMM_F16_ERR_ALIAS;
    const gemm_f16_status st = current_device(dev);
    if (st != GEMM_F16_OK) return st;
    for (const Range& r : in)
        if (r.p && !device_range_ok(r.p, r.bytes)) return GEMM_F16_ERR_INVALID_VALUE;
    if (!device_range_ok(q.c, c_bytes) || (!held && !device_range_ok(q.work, work_bytes))) return GEMM_F16_ERR_INVALID_VALUE;
    return GEMM_F16_OK;
}

gemm_f16_status launch_pair(const Product& q, const Device& dev, const Sizes& sa, const Sizes& sb, cudaStream_t stream)
{
    const bool gated = q.u_codes != nullptr;
    fp8_dev::PairParams p = {};
    p.sw = static_cast<const uint8_t*>(q.b_scales);
    p.su = static_cast<const uint8_t*>(q.u_scales);
    p.sx = static_cast<const uint8_t*>(q.a_scales);
    p.kt = sa.kt, p.w_tiles = sb.row_tiles, p.x_tiles = sa.row_tiles;
    p.group_rows = q.group_rows;
    p.bias = static_cast<const uint16_t*>(q.bias);
    p.C = static_cast<uint16_t*>(q.c);
    p.ldc = q.ldc, p.rows = q.m, p.n = q.n;
    p.groups = static_cast<int32_t>(std::max<int64_t>(q.groups, 1));
    const int64_t tiles_w = cdiv(q.n, gated ? 128 : 256), tiles = (cdiv(q.m, 32) + p.groups) * tiles_w;
    if (tiles > INT32_MAX - 4096) return GEMM_F16_ERR_INVALID_VALUE;   // (an upper bound of their number; they are stepped through)
    p.tiles_w = static_cast<int32_t>(tiles_w);
    // Weight tiles of at most 32 MB walked together, so that A's rows come from DRAM once
    // (131072 x 7168 x 2048 in 8 groups: 1405 us with 8 tiles, 1349 with all 28).
    p.panel = static_cast<int32_t>(std::min<int64_t>(tiles_w, std::max<int64_t>(8, (int64_t(32) << 20) / (256 * sb.pitch))));
    p.k32 = static_cast<int32_t>(cdiv(q.k, 32));
    p.steps = static_cast<int32_t>(cdiv(q.k, 128));
    p.act = q.act;
    p.bf16 = q.dtype == FP8_BF16;
    p.c_unit = 16;   // (and rows of 16-byte units are stored by TMA)
    while (p.c_unit > 2 && ((q.n | q.ldc) * 2 % p.c_unit != 0 || !aligned(q.c, p.c_unit) || (p.c_unit == 16 && q.ldc >> 39)))
        p.c_unit /= 2;
    p.test_stall = option(GEMM_F16_OPT_TEST_STALL) == 1;
    p.timeout_ns = timeout_ns();
    p.status = dev.status;
    const uint32_t box = gated ? 16 : 128;
    if (!encode_codes(&p.tmW, q.b_codes, q.n, p.groups, sb.pitch, box) ||
        (gated && !encode_codes(&p.tmU, q.u_codes, q.n, p.groups, sb.pitch, box)))
        return GEMM_F16_ERR_LAUNCH;
    if (p.c_unit == 16 && !encode_out(&p.tmC, q.c, q.m, q.n, q.ldc, gated)) return GEMM_F16_ERR_LAUNCH;
    const auto kernel = gated ? fp8_dev::gemm_fp8_pair<true> : fp8_dev::gemm_fp8_pair<false>;
    if (!allow_smem(reinterpret_cast<const void*>(kernel), gated ? 1 : 2, fp8_dev::kPairSmem)) return GEMM_F16_ERR_LAUNCH;
    const int64_t clusters = std::min<int64_t>(dev.sms / 2, tiles);
    // Unless it is forced: with groups the kernel finds the width, by the same rule.
    p.width = static_cast<int32_t>(std::min<int64_t>(option(GEMM_F16_OPT_TILE_N), fp8_dev::kMaxWidth));
    if (!q.groups) {
        const int rows = static_cast<int>(q.m);
        int64_t best = p.width ? 0 : INT64_MAX;
        for (int w = fp8_dev::kMaxWidth; w && best; w -= 32) {
            const int parts = fp8_dev::parts_of(rows, w);
            const int64_t cost = fp8_dev::cost_of(static_cast<int>(parts * tiles_w), fp8_dev::width_of(rows, parts),
                                                  static_cast<int>(clusters), p.steps);
            if (cost < best) best = cost, p.width = w;
        }
        p.width = fp8_dev::width_of(rows, fp8_dev::parts_of(rows, p.width));
    }
    for (int i = 0; i < 8; ++i)
        if ((q.groups || p.width == 32 * (i + 1)) && !encode_codes(&p.tmX[i], q.a_codes, q.m, 0, sa.pitch, 16u * (i + 1)))
            return GEMM_F16_ERR_LAUNCH;
    return launch_kernel(kernel, dim3(static_cast<unsigned>(2 * clusters)), fp8_dev::kPairThreads, fp8_dev::kPairSmem, 2,
                         stream, p);
}

// The small form: one 128 x bn tile a cluster, K shared out.
gemm_f16_status launch_tile(const Product& q, const Device& dev, const Sizes& sa, bool after_a, cudaStream_t stream)
{
    fp8_dev::TileParams p = {};
    p.swapped = q.m <= 64 && q.m < q.n;
    p.M = p.swapped ? q.n : q.m;
    p.N = p.swapped ? q.m : q.n;
    p.bn = p.N <= 16 ? 16 : p.N <= 32 ? 32 : p.N <= 64 ? 64 : 128;
    p.sfa = static_cast<const uint8_t*>(p.swapped ? q.b_scales : q.a_scales);
    p.sfb = static_cast<const uint8_t*>(p.swapped ? q.a_scales : q.b_scales);
    p.kt = sa.kt;
    p.bias = static_cast<const uint16_t*>(q.bias);
    p.C = static_cast<uint16_t*>(q.c);
    p.ldc = q.ldc;
    p.k32 = static_cast<int32_t>(cdiv(q.k, 32));
    p.steps = static_cast<int32_t>(cdiv(q.k, 128));
    p.act = q.act;
    p.bf16 = q.dtype == FP8_BF16;
    p.timeout_ns = timeout_ns();
    p.status = dev.status;
    p.test_stall = option(GEMM_F16_OPT_TEST_STALL) == 1;
    p.early = after_a && p.swapped && option(GEMM_F16_OPT_PDL) != 1;
    const uint32_t sbytes = fp8_dev::tile_stage_bytes(p.bn);
    // two CTAs an SM, so that one's loads run under the other's last part
    p.stages = static_cast<int32_t>(std::min<int64_t>(16, (kMaxSmem / 2 - 2048) / sbytes));
    p.tmem_cols = p.bn == 128 ? 256 : p.bn == 64 ? 128 : p.bn == 32 ? 64 : 32;
    const int64_t tiles = cdiv(p.M, 128) * cdiv(p.N, p.bn);
    int cluster = 1;
    // CTAs a tile: 1, 2, 4 or 8, as many as the device holds at once while each has 8 steps, 16
    // where a wide tile has fewer than 32: their sums cost 1 to 5 us, more than a short K
    // saves there (16 steps, 512 x 512 x 2048: 6.5 us by one CTA a tile, 9.9 by two, 9.0 by four; 56
    // steps, 64 x 2048 x 7168: 15.5 by two, 11.0 by the four that this gives, 11.1 by eight).
    const int least = p.bn == 16 || p.steps >= 32 ? 8 : 16;
    while (cluster < 8 && tiles * cluster * 2 <= 2 * dev.sms && cluster * 2 * least <= p.steps) cluster *= 2;
    if (tiles * cluster > INT32_MAX) return GEMM_F16_ERR_INVALID_VALUE;
    if (!encode_codes(&p.tmA, p.swapped ? q.b_codes : q.a_codes, p.M, 0, sa.pitch, 128) ||
        !encode_codes(&p.tmB, p.swapped ? q.a_codes : q.b_codes, p.N, 0, sa.pitch, static_cast<uint32_t>(p.bn)))
        return GEMM_F16_ERR_LAUNCH;
    if (!allow_smem(reinterpret_cast<const void*>(fp8_dev::gemm_fp8_tile), 0, kMaxSmem / 2)) return GEMM_F16_ERR_LAUNCH;
    return launch_kernel(fp8_dev::gemm_fp8_tile, dim3(static_cast<unsigned>(tiles * cluster)), fp8_dev::kTileThreads,
                         p.stages * sbytes + 1024, cluster, stream, p);
}

gemm_f16_status product(Product q, cudaStream_t stream)
{
    Sizes sa, sb;
    Device dev;
    gemm_f16_status st = check(q, &sa, &sb, &dev);
    if (st != GEMM_F16_OK) return st;
    const bool after_a = q.a != nullptr;
    if (after_a) {
        uint8_t* scales = static_cast<uint8_t*>(q.work);
        q.a_scales = scales, q.a_codes = scales + sa.scale_bytes;
        st = run_quantize(q.a, q.a_dtype, 0, q.sm, q.sk, scales + sa.scale_bytes, scales, q.m, q.k, 1, sa, dev.sms, stream);
        if (st != GEMM_F16_OK) return st;
    }
    const int64_t pair = option(GEMM_F16_OPT_PAIR);   // (1 never, 2 always)
    // Small tiles, K shared out where it is long, for up to 32 rows or 64 columns (us, small
    // and pair: 16 x 2048 x 7168 8.6, 15.4; 16 x 16384 x 8192 25.1, 26.9; 65536 x 64 x 1024
    // 11.4, 19.7), for up to 64 rows with a long K and not many columns (64 x 2048 x 7168
    // 11.0, 15.7; 64 x 8192 x 8192 17.5, 18.9; but x 16384 29.6, 27.5 and 64 x 7168 x 2048
    // 11.0, 9.5), and where one turn of them takes a short K, 16-byte rows of C given (1024^3
    // 5.0, 7.8; 1536^3 8.3, 9.3; but 3000 x 300 x 300 12.2, 5.9).  Pairs start 2 us later.
    const int64_t steps = cdiv(q.k, 128);
    const bool few = q.m <= 32 || q.n <= 64 || (q.m <= 64 && steps >= 40 && q.n <= 8192),
               small = q.m > 64 && steps <= 16 && cdiv(q.m, 128) * cdiv(q.n, 128) <= dev.sms && q.n % 8 == 0 &&
                       q.ldc % 8 == 0 && aligned(q.c, 16);
    if (!q.groups && (pair == 1 || (pair != 2 && (few || small)))) return launch_tile(q, dev, sa, after_a, stream);
    return launch_pair(q, dev, sa, sb, stream);
}

}  // namespace

extern "C" {

gemm_f16_status fp8_sizes(int64_t rows, int64_t k, int64_t batch, int64_t* code_bytes, int64_t* scale_bytes)
{
    Sizes s;
    if (!code_bytes || !scale_bytes || !sizes_of(rows, k, batch, &s)) return GEMM_F16_ERR_INVALID_VALUE;
    *code_bytes = s.code_bytes;
    *scale_bytes = s.scale_bytes;
    return GEMM_F16_OK;
}

gemm_f16_status fp8_quantize(const void* x, int dtype, int64_t stride_b, int64_t stride_r, int64_t stride_k,
                             void* codes, void* scales, int64_t rows, int64_t k, int64_t batch, cudaStream_t stream)
{
    Sizes s;
    if (!x || !codes || !scales || dtype < FP8_F16 || dtype > FP8_F32 || !sizes_of(rows, k, batch, &s))
        return GEMM_F16_ERR_INVALID_VALUE;
    if (stride_r <= 0 || stride_k <= 0 || stride_b < 0 || batch > kMaxBatch) return GEMM_F16_ERR_INVALID_VALUE;
    const int64_t eb = elem_bytes(dtype);
    if (!aligned(x, eb) || !aligned(codes, 16) || !aligned(scales, 16)) return GEMM_F16_ERR_INVALID_VALUE;
    int64_t ex, bytes;
    if (!view_extent(rows, k, stride_r, stride_k, &ex) || !batch_extent(ex, batch, stride_b, &ex) ||
        __builtin_mul_overflow(ex, eb, &bytes))
        return GEMM_F16_ERR_INVALID_VALUE;
    if (overlaps(codes, s.code_bytes, x, bytes) || overlaps(scales, s.scale_bytes, x, bytes) ||
        overlaps(codes, s.code_bytes, scales, s.scale_bytes))
        return GEMM_F16_ERR_ALIAS;
    Device dev;
    const gemm_f16_status st = current_device(&dev);
    if (st != GEMM_F16_OK) return st;
    if (!device_range_ok(x, bytes) || !device_range_ok(codes, s.code_bytes) || !device_range_ok(scales, s.scale_bytes))
        return GEMM_F16_ERR_INVALID_VALUE;
    return run_quantize(x, dtype, stride_b, stride_r, stride_k, codes, scales, rows, k, batch, s, dev.sms, stream);
}

gemm_f16_status fp8_dequantize(const void* codes, const void* scales, void* y, int dtype, int64_t rows, int64_t k,
                               int64_t batch, cudaStream_t stream)
{
    Sizes s;
    int64_t bytes;
    if (!codes || !scales || !y || dtype < FP8_F16 || dtype > FP8_F32 || !sizes_of(rows, k, batch, &s) ||
        batch > kMaxBatch || __builtin_mul_overflow(rows * k, batch, &bytes) ||
        __builtin_mul_overflow(bytes, elem_bytes(dtype), &bytes))
        return GEMM_F16_ERR_INVALID_VALUE;
    if (!aligned(y, elem_bytes(dtype)) || !aligned(codes, 16) || !aligned(scales, 16)) return GEMM_F16_ERR_INVALID_VALUE;
    if (overlaps(y, bytes, codes, s.code_bytes) || overlaps(y, bytes, scales, s.scale_bytes)) return GEMM_F16_ERR_ALIAS;
    Device dev;
    const gemm_f16_status st = current_device(&dev);
    if (st != GEMM_F16_OK) return st;
    if (!device_range_ok(y, bytes) || !device_range_ok(codes, s.code_bytes) || !device_range_ok(scales, s.scale_bytes))
        return GEMM_F16_ERR_INVALID_VALUE;
    const fp8_dev::DequantParams p{static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(scales), y, rows, k,
                                   s.pitch, s.kt, s.row_tiles, cdiv(k + 7, 256)};
    return dtype == FP8_F16    ? launch_dequantize<__half>(p, batch, stream)
           : dtype == FP8_BF16 ? launch_dequantize<__nv_bfloat16>(p, batch, stream)
                               : launch_dequantize<float>(p, batch, stream);
}

gemm_f16_status gemm_fp8(const void* A_codes, const void* A_scales, const void* B_codes, const void* B_scales,
                         const void* bias, int act, void* C, int dtype, int64_t ldc, int64_t M, int64_t N, int64_t K,
                         cudaStream_t stream)
{
    if (!A_codes || !A_scales) return GEMM_F16_ERR_INVALID_VALUE;
    Product q = {};
    q.a_codes = A_codes, q.a_scales = A_scales, q.b_codes = B_codes, q.b_scales = B_scales, q.bias = bias;
    q.act = act, q.c = C, q.dtype = dtype, q.ldc = ldc, q.m = M, q.n = N, q.k = K;
    return product(q, stream);
}

gemm_f16_status gemm_fp8_a16(const void* A, int a_dtype, int64_t stride_am, int64_t stride_ak, void* work,
                             const void* B_codes, const void* B_scales, const void* bias, int act, void* C, int dtype,
                             int64_t ldc, int64_t M, int64_t N, int64_t K, cudaStream_t stream)
{
    if (!A) return GEMM_F16_ERR_INVALID_VALUE;
    Product q = {};
    q.a = A, q.a_dtype = a_dtype, q.sm = stride_am, q.sk = stride_ak, q.work = work;
    q.b_codes = B_codes, q.b_scales = B_scales, q.bias = bias;
    q.act = act, q.c = C, q.dtype = dtype, q.ldc = ldc, q.m = M, q.n = N, q.k = K;
    return product(q, stream);
}

gemm_f16_status gemm_fp8_grouped(const void* A_codes, const void* A_scales, const void* B_codes, const void* B_scales,
                                 const void* B_up_codes, const void* B_up_scales, const int32_t* group_rows, int act,
                                 void* C, int dtype, int64_t ldc, int64_t rows, int64_t groups, int64_t N, int64_t K,
                                 cudaStream_t stream)
{
    if (rows == 0) return GEMM_F16_OK;
    if (!A_codes || !A_scales || groups < 1) return GEMM_F16_ERR_INVALID_VALUE;
    Product q = {};
    q.a_codes = A_codes, q.a_scales = A_scales, q.b_codes = B_codes, q.b_scales = B_scales;
    q.u_codes = B_up_codes, q.u_scales = B_up_scales, q.group_rows = group_rows;
    q.act = act, q.c = C, q.dtype = dtype, q.ldc = ldc, q.m = rows, q.n = N, q.k = K, q.groups = groups;
    return product(q, stream);
}

gemm_f16_status gemm_fp8_grouped_a16(const void* A, int a_dtype, int64_t stride_am, int64_t stride_ak, void* work,
                                     const void* B_codes, const void* B_scales, const void* B_up_codes,
                                     const void* B_up_scales, const int32_t* group_rows, int act, void* C, int dtype,
                                     int64_t ldc, int64_t rows, int64_t groups, int64_t N, int64_t K,
                                     cudaStream_t stream)
{
    if (rows == 0) return GEMM_F16_OK;
    if (!A || groups < 1) return GEMM_F16_ERR_INVALID_VALUE;
    Product q = {};
    q.a = A, q.a_dtype = a_dtype, q.sm = stride_am, q.sk = stride_ak, q.work = work;
    q.b_codes = B_codes, q.b_scales = B_scales;
    q.u_codes = B_up_codes, q.u_scales = B_up_scales, q.group_rows = group_rows;
    q.act = act, q.c = C, q.dtype = dtype, q.ldc = ldc, q.m = rows, q.n = N, q.k = K, q.groups = groups;
    return product(q, stream);
}

}  // extern "C"
