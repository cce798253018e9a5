// Host side of the MXFP4 entry points (gemm_mxf4.h): argument checks, the
// choice of form, tensor maps and launches.
#include <algorithm>
#include <cstdint>
#include <mutex>

#include "gemm_mxf4.h"
#include "host.h"
#include "mxf4_convert.cuh"
#include "mxf4_gemm.cuh"

using namespace gemm_f16_host;

namespace {

constexpr int kMaxSmem = 232448;

struct Sizes {
    int64_t blocks, pitch, kt, row_tiles, code_bytes, scale_bytes;   // bytes of the whole batch
};

bool sizes_of(int64_t rows, int64_t k, int64_t batch, Sizes* s)
{
    if (rows < 1 || k < 1 || batch < 1 || rows > GEMM_F16_MAX_DIM || k > GEMM_F16_MAX_DIM) return false;
    s->blocks = cdiv(k, 32);
    s->pitch = s->blocks * 16;
    s->kt = cdiv(s->blocks, 4);
    s->row_tiles = cdiv(rows, 128);
    if (__builtin_mul_overflow(rows * s->pitch, batch, &s->code_bytes)) return false;
    return !__builtin_mul_overflow(s->row_tiles * s->kt * mxf4_dev::kScaleTile, batch, &s->scale_bytes);
}

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

int64_t elem_bytes(int dtype) { return dtype == MXF4_F32 ? 4 : 2; }

// Batches are the third grid dimension.
constexpr int64_t kMaxBatch = 65535;

bool encode_codes(CUtensorMap* tm, const void* codes, int64_t rows, int64_t pitch, uint32_t box_rows)
{
    const auto encode = tensor_map_encoder();
    if (!encode) return false;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(pitch), static_cast<cuuint64_t>(rows)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(pitch)};
    cuuint32_t box[2] = {128, box_rows};
    cuuint32_t estr[2] = {1, 1};
    return encode(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(codes), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T>
gemm_f16_status launch_quantize(const mxf4_dev::QuantParams& p, int64_t batch, cudaStream_t stream)
{
    const int64_t tiles = p.row_tiles * p.col_tiles;
    if (tiles > INT32_MAX) return GEMM_F16_ERR_INVALID_VALUE;
    const dim3 grid(static_cast<unsigned>(tiles), 1, static_cast<unsigned>(batch));
    const bool vec = aligned(p.x, 16) && p.sr * sizeof(T) % 16 == 0 && p.sb * sizeof(T) % 16 == 0;
    const auto kernel = p.sk != 1 ? mxf4_dev::quantize_strided<T>
                        : vec     ? mxf4_dev::quantize_rows<T, true>
                                  : mxf4_dev::quantize_rows<T, false>;
    return launch_kernel(kernel, grid, mxf4_dev::kConvThreads, 0, 1, stream, p);
}

template <typename T>
gemm_f16_status launch_dequantize(const mxf4_dev::DequantParams& p, int64_t batch, cudaStream_t stream)
{
    const int64_t blocks = cdiv(p.rows, mxf4_dev::kDequantRows) * p.col_tiles;
    if (blocks > INT32_MAX) return GEMM_F16_ERR_INVALID_VALUE;
    const dim3 grid(static_cast<unsigned>(blocks), 1, static_cast<unsigned>(batch));
    return launch_kernel(p.k % 8 == 0 && aligned(p.y, 16) ? mxf4_dev::dequantize<T, true> : mxf4_dev::dequantize<T, false>,
                         grid, mxf4_dev::kConvThreads, 0, 1, stream, p);
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

// Checks of a product's operands but A; `work`: bytes of A's buffers that C and
// the inputs must keep out of.
gemm_f16_status check_product(const void* B_codes, const void* B_scales, const void* bias, int act, const void* C,
                              int64_t ldc, int64_t M, int64_t N, int64_t K, Sizes* sa, Sizes* sb, int64_t* c_bytes)
{
    int64_t ec;
    if (!B_codes || !B_scales || !C || !sizes_of(M, K, 1, sa) || !sizes_of(N, K, 1, sb)) return GEMM_F16_ERR_INVALID_VALUE;
    if (act < GEMM_F16_ACT_NONE || act > GEMM_F16_ACT_GELU || ldc < N || !view_extent(M, N, ldc, 1, &ec) ||
        __builtin_mul_overflow(ec, 2, c_bytes))
        return GEMM_F16_ERR_INVALID_VALUE;
    if (!aligned(B_codes, 16) || !aligned(B_scales, 16) || !aligned(C, 2) || !aligned(bias, 2))
        return GEMM_F16_ERR_INVALID_VALUE;
    if (overlaps(C, *c_bytes, B_codes, sb->code_bytes) || overlaps(C, *c_bytes, B_scales, sb->scale_bytes) ||
        (bias && overlaps(C, *c_bytes, bias, 2 * N)))
        return GEMM_F16_ERR_ALIAS;
    return GEMM_F16_OK;
}

bool product_memory_ok(const void* B_codes, const void* B_scales, const void* bias, const void* C, int64_t N,
                       const Sizes& sb, int64_t c_bytes)
{
    return device_range_ok(B_codes, sb.code_bytes) && device_range_ok(B_scales, sb.scale_bytes) &&
           device_range_ok(C, c_bytes) && (!bias || device_range_ok(bias, 2 * N));
}

gemm_f16_status run_quantize(const void* x, int dtype, int64_t sb, int64_t sr, int64_t sk, void* codes, void* scales,
                             int64_t rows, int64_t k, int64_t batch, const Sizes& s, cudaStream_t stream)
{
    const mxf4_dev::QuantParams p{x, sb, sr, sk, static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales), rows, k,
                                  s.pitch, s.kt, s.row_tiles, cdiv(k, sk == 1 ? mxf4_dev::kTileVals : mxf4_dev::kStridedVals)};
    return dtype == MXF4_F16    ? launch_quantize<__half>(p, batch, stream)
           : dtype == MXF4_BF16 ? launch_quantize<__nv_bfloat16>(p, batch, stream)
                                : launch_quantize<float>(p, batch, stream);
}

// Scale tiles as rows of 128 words, two a box.
bool encode_scales(CUtensorMap* tm, const void* scales, int64_t tiles)
{
    const auto encode = tensor_map_encoder();
    if (!encode) return false;
    cuuint64_t dims[2] = {128, static_cast<cuuint64_t>(tiles)};
    cuuint64_t strides[1] = {mxf4_dev::kScaleTile};
    cuuint32_t box[2] = {128, 2};
    cuuint32_t estr[2] = {1, 1};
    return encode(tm, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void*>(scales), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_out(CUtensorMap* tm, void* C, int64_t M, int64_t N, int64_t ldc)
{
    const auto encode = tensor_map_encoder();
    if (!encode) return false;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(M)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(2 * ldc)};
    cuuint32_t box[2] = {64, 32};
    cuuint32_t estr[2] = {1, 1};
    return encode(tm, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, C, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

// C's rows can be stored by TMA, which clips a box to whole 16 bytes.
bool tma_rows(const void* C, int64_t ldc, int64_t N)
{
    return N % 8 == 0 && ldc % 8 == 0 && ldc < int64_t(1) << 39 && aligned(C, 16);
}

template <int kBN>
gemm_f16_status launch_pair(const Device& dev, const void* A_codes, const void* A_scales, const void* B_codes,
                            const void* B_scales, const void* bias, int act, void* C, int64_t ldc, int64_t M, int64_t N,
                            int64_t K, cudaStream_t stream)
{
    using Shape = mxf4_dev::PairShape<kBN>;
    Sizes sa, sb;
    sizes_of(M, K, 1, &sa);
    sizes_of(N, K, 1, &sb);
    mxf4_dev::PairParams p = {};
    p.bias = static_cast<const __half*>(bias);
    p.C = static_cast<__half*>(C);
    p.ldc = ldc, p.M = M, p.N = N;
    p.kt = static_cast<int32_t>(sa.kt);
    p.k64 = static_cast<int32_t>(cdiv(K, 64));
    p.steps = static_cast<int32_t>(cdiv(K, 256));
    p.act = act;
    p.tiles_m = static_cast<int32_t>(cdiv(M, 256));
    p.tiles_n = static_cast<int32_t>(cdiv(N, kBN));
    p.panel = p.tiles_n <= 16 ? 2 : 8;
    p.test_stall = option(GEMM_F16_OPT_TEST_STALL) == 1;
    p.timeout_ns = timeout_ns();
    p.status = dev.status;
    p.c_tma = tma_rows(C, ldc, N);
    if (!encode_codes(&p.tmA, A_codes, M, sa.pitch, 128) || !encode_codes(&p.tmB, B_codes, N, sa.pitch, kBN / 2) ||
        !encode_scales(&p.tmSA, A_scales, sa.row_tiles * sa.kt) || !encode_scales(&p.tmSB, B_scales, sb.row_tiles * sb.kt) ||
        (p.c_tma && !encode_out(&p.tmC, C, M, N, ldc)))
        return GEMM_F16_ERR_LAUNCH;
    if (!allow_smem(reinterpret_cast<const void*>(mxf4_dev::gemm_mxf4_pair<kBN>), kBN == 256 ? 1 : 2, Shape::kSmem))
        return GEMM_F16_ERR_LAUNCH;
    const int64_t clusters = std::min<int64_t>(dev.sms / 2, static_cast<int64_t>(p.tiles_m) * p.tiles_n);
    return launch_kernel(mxf4_dev::gemm_mxf4_pair<kBN>, dim3(static_cast<unsigned>(2 * clusters)), mxf4_dev::kPairThreads,
                         Shape::kSmem, 2, stream, p);
}

// The product of checked operands; `after_a`: the kernel before is this call's
// quantisation of A.
gemm_f16_status product(const Device& dev, const void* A_codes, const void* A_scales, const void* B_codes,
                        const void* B_scales, const void* bias, int act, void* C, int64_t ldc, int64_t M, int64_t N,
                        int64_t K, bool after_a, cudaStream_t stream)
{
    Sizes sa;
    sizes_of(M, K, 1, &sa);
    // Pairs, but for few tiles with a long K, which small tiles share out: a pair takes
    // 3.7 us and 0.22 a step, the split form 12 us until its own steps count (1024^3: 4.6
    // and 11.3 us; 96 x 4096 x 4096: 7.0, 14.9; 128 x 2048 x 8192: 10.6, 12.3; 2048^3: 7.3,
    // 8.4; 128 x 8192 x 8192: 11.3, 14.1).
    // Of the two widths the one whose turns of the clusters cost less: a
    // 128-wide turn takes 0.72 of a 256-wide one (16384 x 2048 x 7168: 14 turns in 97 us, 7 in
    // 68 us), 0.62 where rows are stored without TMA and the last turn's stores, which nothing
    // hides, are longer (3001 x 2000 x 4097, two turns of 256 or three of 128: 18.0 us, 18.8 us;
    // x 1999: 25.1 us, 23.3 us).
    const int64_t pairs = dev.sms / 2, wide = cdiv(M, 256) * cdiv(N, 256), narrow = cdiv(M, 256) * cdiv(N, 128);
    const double turn = tma_rows(C, ldc, N) ? 0.72 : 0.62;
    const bool split = narrow * 4 < pairs * 3 && cdiv(K, 256) > 40;
    if (M > 64 && N > 64 && !split && sa.row_tiles * sa.kt < INT32_MAX && cdiv(N, 128) * sa.kt < INT32_MAX)
        return cdiv(narrow, pairs) * turn < cdiv(wide, pairs)
                   ? launch_pair<128>(dev, A_codes, A_scales, B_codes, B_scales, bias, act, C, ldc, M, N, K, stream)
                   : launch_pair<256>(dev, A_codes, A_scales, B_codes, B_scales, bias, act, C, ldc, M, N, K, stream);
    mxf4_dev::GemmParams p = {};
    // Few rows of A: B's rows take the 128 lanes and A's rows the narrow side, as narrow as
    // they fit (16 x 16384 x 8192: 10.1 us, 18.3 with 64 columns, 23.2 the other way round;
    // 64 x 8192 x 8192: 11.0 us, 13.5 the other way round); the same for few columns
    // (65536 x 16 x 7168: 41 us, 59 with 128 columns).
    p.swapped = M <= 64 && M < N;
    p.M = p.swapped ? N : M;
    p.N = p.swapped ? M : N;
    p.bn = p.N <= 16 ? 16 : p.N <= 32 ? 32 : p.N <= 64 ? 64 : 128;
    p.sfa = static_cast<const uint8_t*>(p.swapped ? B_scales : A_scales);
    p.sfb = static_cast<const uint8_t*>(p.swapped ? A_scales : B_scales);
    p.kt = sa.kt;
    p.bias = static_cast<const __half*>(bias);
    p.C = static_cast<__half*>(C);
    p.ldc = ldc;
    p.k64 = static_cast<int32_t>(cdiv(K, 64));
    p.steps = static_cast<int32_t>(cdiv(K, 256));
    p.act = act;
    p.timeout_ns = timeout_ns();
    p.status = dev.status;
    p.test_stall = option(GEMM_F16_OPT_TEST_STALL) == 1;
    p.early = after_a && p.swapped && option(GEMM_F16_OPT_PDL) != 1;
    const uint32_t sbytes = mxf4_dev::gemm_stage_bytes(p.bn);
    // two CTAs an SM, so that one's loads run under the other's last part
    p.stages = static_cast<int32_t>(std::min<int64_t>(16, (kMaxSmem / 2 - 2048) / sbytes));
    p.tmem_cols = p.bn == 128 ? 256 : p.bn == 64 ? 128 : p.bn == 32 ? 64 : 32;
    const int64_t tiles = cdiv(p.M, 128) * cdiv(p.N, p.bn);
    // As many CTAs a tile as the device holds at once, while each has 8 steps: their sums
    // cost 1 to 2 us (1 x 2048 x 2048, 8 steps: 4.7 us by one CTA, 5.9 by 4, 7.0 by 8;
    // 16 x 4096 x 8192, 32 steps: 11.1, 7.6, 8.8; 16 x 2048 x 16384, 64 steps: 19.0, 9.4, 8.9).
    int cluster = 1;
    while (cluster < 8 && tiles * cluster * 2 <= 2 * dev.sms && cluster * 16 <= p.steps) cluster *= 2;
    if (tiles * cluster > INT32_MAX) return GEMM_F16_ERR_INVALID_VALUE;
    if (!encode_codes(&p.tmA, p.swapped ? B_codes : A_codes, p.M, sa.pitch, 128) ||
        !encode_codes(&p.tmB, p.swapped ? A_codes : B_codes, p.N, sa.pitch, static_cast<uint32_t>(p.bn)))
        return GEMM_F16_ERR_LAUNCH;
    if (!allow_smem(reinterpret_cast<const void*>(mxf4_dev::gemm_mxf4_tile), 0, kMaxSmem / 2)) return GEMM_F16_ERR_LAUNCH;
    return launch_kernel(mxf4_dev::gemm_mxf4_tile, dim3(static_cast<unsigned>(tiles * cluster)), mxf4_dev::kGemmThreads,
                         p.stages * sbytes + 1024, cluster, stream, p);
}

}  // namespace

extern "C" {

gemm_f16_status mxf4_sizes(int64_t rows, int64_t k, int64_t batch, int64_t* code_bytes, int64_t* scale_bytes)
{
    Sizes s;
    if (!code_bytes || !scale_bytes || !sizes_of(rows, k, batch, &s)) return GEMM_F16_ERR_INVALID_VALUE;
    *code_bytes = s.code_bytes;
    *scale_bytes = s.scale_bytes;
    return GEMM_F16_OK;
}

gemm_f16_status mxf4_quantize(const void* x, int dtype, int64_t stride_b, int64_t stride_r, int64_t stride_k,
                              void* codes, void* scales, int64_t rows, int64_t k, int64_t batch, cudaStream_t stream)
{
    Sizes s;
    if (!x || !codes || !scales || dtype < MXF4_F16 || dtype > MXF4_F32 || !sizes_of(rows, k, batch, &s))
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
    return run_quantize(x, dtype, stride_b, stride_r, stride_k, codes, scales, rows, k, batch, s, stream);
}

gemm_f16_status mxf4_dequantize(const void* codes, const void* scales, void* y, int dtype, int64_t rows, int64_t k,
                                int64_t batch, cudaStream_t stream)
{
    Sizes s;
    int64_t bytes;
    if (!codes || !scales || !y || dtype < MXF4_F16 || dtype > MXF4_F32 || !sizes_of(rows, k, batch, &s) ||
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
    const mxf4_dev::DequantParams p{static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(scales), y, rows, k,
                                    s.pitch, s.kt, s.row_tiles, cdiv(k + 7, mxf4_dev::kTileVals)};
    return dtype == MXF4_F16    ? launch_dequantize<__half>(p, batch, stream)
           : dtype == MXF4_BF16 ? launch_dequantize<__nv_bfloat16>(p, batch, stream)
                                : launch_dequantize<float>(p, batch, stream);
}

gemm_f16_status gemm_mxf4(const void* A_codes, const void* A_scales, const void* B_codes, const void* B_scales,
                          const void* bias, int act, void* C, int64_t ldc, int64_t M, int64_t N, int64_t K,
                          cudaStream_t stream)
{
    Sizes sa, sb;
    int64_t bytes;
    if (!A_codes || !A_scales || !aligned(A_codes, 16) || !aligned(A_scales, 16)) return GEMM_F16_ERR_INVALID_VALUE;
    gemm_f16_status st = check_product(B_codes, B_scales, bias, act, C, ldc, M, N, K, &sa, &sb, &bytes);
    if (st != GEMM_F16_OK) return st;
    if (overlaps(C, bytes, A_codes, sa.code_bytes) || overlaps(C, bytes, A_scales, sa.scale_bytes))
        return GEMM_F16_ERR_ALIAS;
    Device dev;
    st = current_device(&dev);
    if (st != GEMM_F16_OK) return st;
    if (!device_range_ok(A_codes, sa.code_bytes) || !device_range_ok(A_scales, sa.scale_bytes) ||
        !product_memory_ok(B_codes, B_scales, bias, C, N, sb, bytes))
        return GEMM_F16_ERR_INVALID_VALUE;
    return product(dev, A_codes, A_scales, B_codes, B_scales, bias, act, C, ldc, M, N, K, false, stream);
}

gemm_f16_status gemm_mxf4_a16(const void* A, int64_t stride_am, int64_t stride_ak, void* work, const void* B_codes,
                              const void* B_scales, const void* bias, int act, void* C, int64_t ldc, int64_t M,
                              int64_t N, int64_t K, cudaStream_t stream)
{
    Sizes sa, sb;
    int64_t bytes, ea;
    if (!A || !work || !aligned(A, 2) || !aligned(work, 16) || stride_am <= 0 || stride_ak <= 0)
        return GEMM_F16_ERR_INVALID_VALUE;
    gemm_f16_status st = check_product(B_codes, B_scales, bias, act, C, ldc, M, N, K, &sa, &sb, &bytes);
    if (st != GEMM_F16_OK) return st;
    if (!view_extent(M, K, stride_am, stride_ak, &ea) || __builtin_mul_overflow(ea, 2, &ea))
        return GEMM_F16_ERR_INVALID_VALUE;
    const int64_t wb = sa.code_bytes + sa.scale_bytes;
    if (overlaps(C, bytes, A, ea) || overlaps(C, bytes, work, wb) || overlaps(work, wb, A, ea) ||
        overlaps(work, wb, B_codes, sb.code_bytes) || overlaps(work, wb, B_scales, sb.scale_bytes) ||
        (bias && overlaps(work, wb, bias, 2 * N)))
        return GEMM_F16_ERR_ALIAS;
    Device dev;
    st = current_device(&dev);
    if (st != GEMM_F16_OK) return st;
    if (!device_range_ok(A, ea) || !device_range_ok(work, wb) || !product_memory_ok(B_codes, B_scales, bias, C, N, sb, bytes))
        return GEMM_F16_ERR_INVALID_VALUE;
    uint8_t* scales = static_cast<uint8_t*>(work);
    uint8_t* codes = scales + sa.scale_bytes;
    st = run_quantize(A, MXF4_F16, 0, stride_am, stride_ak, codes, scales, M, K, 1, sa, stream);
    if (st != GEMM_F16_OK) return st;
    return product(dev, codes, scales, B_codes, B_scales, bias, act, C, ldc, M, N, K, true, stream);
}

}  // extern "C"
