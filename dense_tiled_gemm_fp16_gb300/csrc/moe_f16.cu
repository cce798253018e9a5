// Host side of the mixture-of-experts layer (moe_f16.h): argument checks, the
// workspace and the two launches.
#include <algorithm>
#include <cstdint>
#include <mutex>

#include "gemm_mxf4.h"
#include "host.h"
#include "moe_f16.h"
#include "moe_kernel.cuh"
#include "moe_stream.cuh"

using namespace gemm_f16_host;

static_assert(MOE_F16_MAX_TOKENS == moe_dev::kMaxTokens && MOE_F16_MAX_EXPERTS == moe_dev::kMaxExperts &&
                  MOE_F16_MAX_TOP_K == moe_dev::kMaxTop,
              "the header and the kernels agree on the limits");

namespace {

int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }
bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// The counters at the workspace's start.
constexpr int64_t kControlBytes = 8448;
static_assert(sizeof(moe_dev::StreamControl) <= kControlBytes && 256 + moe_dev::kMaxRanges * 4 <= kControlBytes, "room");

// Places in the workspace.
struct Layout {
    int64_t dp, fp, xp, hp, parts, bytes;              // any format
    int64_t dq, fq, dw, fw, xq, xs, hq, hs;            // MXFP4 columns: row pitches of codes and of scales
};

bool layout_of(int64_t T, int64_t D, int64_t F, int64_t E, int64_t top, Layout* l)
{
    if (T < 1 || T > MOE_F16_MAX_TOKENS || E < 1 || E > MOE_F16_MAX_EXPERTS || top < 1 || top > MOE_F16_MAX_TOP_K ||
        top > E || D < 1 || D > MOE_F16_MAX_DIM || F < 1 || F > MOE_F16_MAX_DIM)
        return false;
    l->dp = round_up(D, 64);
    l->fp = round_up(F, 64);
    l->dq = round_up(D, 256) / 2, l->fq = round_up(F, 256) / 2;
    l->dw = round_up(D, 256) / 32, l->fw = round_up(F, 256) / 32;
    int64_t at = kControlBytes;
    auto take = [&](int64_t bytes) {
        const int64_t place = at;
        at += round_up(bytes, 256);
        return place;
    };
    l->xp = take(T * l->dp * 2);
    l->hp = take(T * top * 2 * l->fp * 2);
    l->xq = take(T * moe_dev::kPieces * l->dq);
    l->xs = take(T * moe_dev::kPieces * l->dw);
    l->hq = take(T * top * moe_dev::kPieces * l->fq);
    l->hs = take(T * top * moe_dev::kPieces * l->fw);
    l->parts = take(std::max(moe_dev::kMaxSplits * T * l->dp * 4,
                             static_cast<int64_t>(moe_dev::kMaxParts) * 2 * std::max<int64_t>(T, 16) * 256 * 4));
    l->bytes = at;
    return true;
}

// Bytes that one projection spans; false where the description is not valid.
bool weight_span(const moe_f16_weight& w, int64_t E, int64_t in, int64_t out, int64_t* data, int64_t* scales)
{
    if (!w.data) return false;
    if (w.format == MOE_F16_WEIGHT_MXF4)
        return w.scales && aligned(w.data, 16) && aligned(w.scales, 16) &&
               mxf4_sizes(out, in, E, data, scales) == GEMM_F16_OK;
    if (w.format != MOE_F16_WEIGHT_F16 || w.scales || !aligned(w.data, 2)) return false;
    if (w.stride_e < 0 || w.stride_i <= 0 || w.stride_o <= 0) return false;
    int64_t e;
    if (!view_extent(in, out, w.stride_i, w.stride_o, &e) || !batch_extent(e, E, w.stride_e, &e)) return false;
    *scales = 0;
    return !__builtin_mul_overflow(e, 2, data);
}

// What a tensor map can address: unit stride along one matrix axis, the other
// strides positive multiples of 16 bytes below 2^40, an aligned start.
bool map_strides(const moe_f16_weight& w, int64_t pitch, int64_t E)
{
    return pitch % 8 == 0 && pitch < int64_t(1) << 39 && aligned(w.data, 16) &&
           (E == 1 || (w.stride_e > 0 && w.stride_e % 8 == 0 && w.stride_e < int64_t(1) << 39));
}

bool rows_aligned(const moe_f16_weight& w, int64_t E) { return w.stride_i == 1 && map_strides(w, w.stride_o, E); }
bool cols_aligned(const moe_f16_weight& w, int64_t E) { return w.stride_o == 1 && map_strides(w, w.stride_i, E); }

moe_dev::Weight weight_of(const moe_f16_weight& w, int64_t E, int64_t in, int64_t out)
{
    moe_dev::Weight r = {};
    r.data = static_cast<const uint8_t*>(w.data);
    r.scales = static_cast<const uint8_t*>(w.scales);
    if (w.format == MOE_F16_WEIGHT_MXF4) {
        int64_t code, scale;
        mxf4_sizes(out, in, 1, &code, &scale);
        r.so = code / out;
        r.se = code;
        r.scale_se = scale;
        r.kt = static_cast<int32_t>(cdiv(in, 128));
    } else {
        r.se = w.stride_e, r.si = w.stride_i, r.so = w.stride_o;
    }
    return r;
}

constexpr int kMaxDevices = 64;
constexpr int kMaxSmem = 232448;     // 227 KiB a block
constexpr int kStaticSmem = 9216;    // more than the stream kernel's own

// More dynamic shared memory than the default, once a device and kernel.
bool allow_smem(const void* kernel, int slot, int bytes)
{
    static std::mutex mutex;
    static int have[kMaxDevices][32] = {};
    int d = 0;
    if (cudaGetDevice(&d) != cudaSuccess || d < 0 || d >= kMaxDevices) {
        cudaGetLastError();
        return false;
    }
    std::lock_guard<std::mutex> lk(mutex);
    if (have[d][slot] >= bytes) return true;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    have[d][slot] = bytes;
    return true;
}

template <int kLayout, int kPer>
gemm_f16_status launch_route(const moe_dev::Params& p, cudaStream_t stream)
{
    const int smem = moe_dev::RouteShape(p.dp, p.E, kLayout == moe_dev::kOutContiguous).bytes;
    const auto kernel = moe_dev::moe_route<kLayout, kPer>;
    if (!allow_smem(reinterpret_cast<const void*>(kernel), 2 * kLayout + (kPer > 2), smem)) return GEMM_F16_ERR_LAUNCH;
    const unsigned groups = static_cast<unsigned>((p.T + 7) / 8);
    return launch_kernel(kernel, dim3(groups * moe_dev::kRouteCluster), moe_dev::kThreads, smem, moe_dev::kRouteCluster,
                         stream, p);
}

// Up to 64 experts the choosing warp's code is short: with the form for 512, 64 experts took
// 47.8 us instead of 42.3 (4 tokens, MXFP4) and 8 experts 78.2 instead of 74.9 (1 token, fp16).
template <int kLayout>
gemm_f16_status launch_route(const moe_dev::Params& p, cudaStream_t stream)
{
    return p.E <= 64 ? launch_route<kLayout, 2>(p, stream) : launch_route<kLayout, moe_dev::kMaxExperts / 32>(p, stream);
}

template <int kFmt, int kGroups, int kRing>
gemm_f16_status launch_experts(moe_dev::Params& p, int sms, cudaStream_t stream)
{
    constexpr int kOut = moe_dev::Step<kFmt, false>::kOut;
    // The count that leaves the fewest idle parts in the last turn of the CTAs.
    const int64_t ranges = cdiv(p.D, kOut);
    p.splits = 1;
    double best = 0;
    for (int s = 1; s <= moe_dev::kMaxSplits; ++s) {
        const double fill = static_cast<double>(ranges * s) / (cdiv(ranges * s, sms) * sms);
        if (fill > best + 0.04) best = fill, p.splits = s;
    }
    const int ring = moe_dev::kWarps * kRing * moe_dev::kStepBytes;
    const int smem = ring + std::max(2 * moe_dev::kWarps * kGroups * 32 * 16, moe_dev::kWarps * p.T * kOut * 4);
    const auto kernel = moe_dev::moe_experts<kFmt, kGroups, kRing>;
    if (!allow_smem(reinterpret_cast<const void*>(kernel), 16 + 4 * kFmt + (kGroups > 1) + 2 * (kRing == 2), smem))
        return GEMM_F16_ERR_LAUNCH;
    return launch_kernel(kernel, dim3(static_cast<unsigned>(sms)), moe_dev::kThreads, smem, 1, stream, p);
}

// Pieces of 8 tokens an expert, or of 16 when there are more than 8 in all (8 of 64
// experts of 2047 x 1023: 1 token 72 us, 78 with pieces of 16; 8 tokens 196, 221).
template <int kFmt, int kRing>
gemm_f16_status launch_experts(moe_dev::Params& p, int sms, cudaStream_t stream)
{
    if (p.T <= 8) return launch_experts<kFmt, 1, kRing>(p, sms, stream);
    // (32-column ranges of more than 32 tokens: the sums take the ring's room)
    if constexpr (kFmt == moe_dev::kF16Cols) {
        if (p.T > 32) return launch_experts<kFmt, 2, 2>(p, sms, stream);
    }
    return launch_experts<kFmt, 2, kRing>(p, sms, stream);
}

// A 3-D map of one projection: inner, outer, expert; boxes of 128 bytes x rows.
// The L2 brings 256 bytes of a row where the next step reads the other half,
// 128 where that is another unit's.
bool encode_weight(CUtensorMap* tm, const void* data, bool bytes, uint32_t box_rows, bool along_k, uint64_t inner,
                   uint64_t outer, uint64_t experts, uint64_t pitch, uint64_t expert_pitch)
{
    const auto encode = tensor_map_encoder();
    if (!encode) return false;
    cuuint64_t dims[3] = {inner, outer, experts};
    cuuint64_t strides[2] = {pitch, experts > 1 ? expert_pitch : pitch * outer};
    cuuint32_t box[3] = {bytes ? 128u : 64u, box_rows, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return encode(tm, bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(data),
                  dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  along_k ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int kFmt>
gemm_f16_status launch_stream(const moe_dev::Params& p, const Layout& l, uint8_t* ws, const moe_f16_weight* const* w,
                              int sms, cudaStream_t stream)
{
    constexpr bool kMx = kFmt == moe_dev::kStreamMxf4;
    moe_dev::StreamParams sp = {};
    sp.p = p;
    CUtensorMap* maps[3] = {&sp.gate, &sp.up, &sp.down};
    const moe_dev::Weight* dw[3] = {&p.gate, &p.up, &p.down};
    for (int i = 0; i < 3; ++i) {
        const uint64_t in = i < 2 ? p.D : p.F, out = i < 2 ? p.F : p.D;
        const bool good =
            kMx ? encode_weight(maps[i], w[i]->data, true, 128, true, dw[i]->so, out, p.E, dw[i]->so, dw[i]->se)
            : kFmt == moe_dev::kStreamRows
                ? encode_weight(maps[i], w[i]->data, false, 128, true, in, out, p.E, 2 * dw[i]->so, 2 * dw[i]->se)
                : encode_weight(maps[i], w[i]->data, false, 64, false, out, in, p.E, 2 * dw[i]->si, 2 * dw[i]->se);
        if (!good) return GEMM_F16_ERR_LAUNCH;
    }
    sp.ctl = reinterpret_cast<moe_dev::StreamControl*>(ws);
    sp.sums = reinterpret_cast<float*>(ws + l.parts);
    sp.x = kMx ? ws + l.xq : ws + l.xp;
    sp.xs = ws + l.xs;
    sp.h = kMx ? ws + l.hq : ws + l.hp;
    sp.hs = ws + l.hs;
    sp.xpitch = static_cast<int32_t>(kMx ? l.dq : 2 * l.dp);
    sp.hpitch = static_cast<int32_t>(kMx ? l.fq : 2 * l.fp);
    sp.xwords = static_cast<int32_t>(l.dw / 4);
    sp.hwords = static_cast<int32_t>(l.fw / 4);
    const moe_dev::StreamShape shape(kMx, p.T);
    sp.cap = shape.cap;
    sp.b_bytes = static_cast<int32_t>((kMx ? sp.cap * moe_dev::kPieces : 2 * sp.cap) * 128);
    sp.stage_bytes = 2 * static_cast<int32_t>(moe_dev::kTileBytes) + sp.b_bytes + (kMx ? 6 * mxf4_dev::kScaleTile : 0);
    sp.stages = std::min(16, (kMaxSmem - kStaticSmem - 1024) / sp.stage_bytes);
    sp.acc_cols = shape.acc_cols;
    sp.y_col = shape.y_col;
    sp.tmem_cols = shape.alloc;
    const int smem = sp.stages * sp.stage_bytes + 1024;
    const auto kernel = moe_dev::moe_stream<kFmt>;
    if (!allow_smem(reinterpret_cast<const void*>(kernel), 12 + kFmt, kMaxSmem - kStaticSmem)) return GEMM_F16_ERR_LAUNCH;
    return launch_kernel(kernel, dim3(static_cast<unsigned>(std::min(sms, moe_dev::kMaxParts))), moe_dev::kThreads, smem, 1,
                         stream, sp);
}

}  // namespace

extern "C" {

gemm_f16_status moe_f16_workspace_size(int64_t T, int64_t D, int64_t F, int64_t E, int64_t top_k, size_t* bytes)
{
    Layout l;
    if (!bytes || !layout_of(T, D, F, E, top_k, &l)) return GEMM_F16_ERR_INVALID_VALUE;
    *bytes = static_cast<size_t>(l.bytes);
    return GEMM_F16_OK;
}

gemm_f16_status moe_f16(const void* x, int64_t stride_xt, int64_t stride_xi, const void* router, int64_t stride_ri,
                        int64_t stride_re, const moe_f16_weight* gate, const moe_f16_weight* up,
                        const moe_f16_weight* down, int64_t T, int64_t D, int64_t F, int64_t E, int64_t top_k,
                        int renormalize, int act, void* y, int64_t ldy, float* weights, int32_t* ids, void* workspace,
                        size_t workspace_bytes, cudaStream_t stream)
{
    Layout l;
    if (!x || !router || !gate || !up || !down || !y || !weights || !ids || !workspace || !layout_of(T, D, F, E, top_k, &l))
        return GEMM_F16_ERR_INVALID_VALUE;
    if (stride_xt <= 0 || stride_xi <= 0 || stride_ri <= 0 || stride_re <= 0 || ldy < D || act < GEMM_F16_ACT_NONE ||
        act > GEMM_F16_ACT_GELU || gate->format != up->format || gate->format != down->format)
        return GEMM_F16_ERR_INVALID_VALUE;
    if (!aligned(x, 2) || !aligned(router, 2) || !aligned(y, 2) || !aligned(weights, 4) || !aligned(ids, 4) ||
        !aligned(workspace, 256))
        return GEMM_F16_ERR_INVALID_VALUE;
    struct Span {
        const void* p;
        int64_t bytes;
    };
    Span in[8], out[4];
    int nin = 0, nout = 0;
    int64_t e;
    if (!view_extent(T, D, stride_xt, stride_xi, &e) || __builtin_mul_overflow(e, 2, &e)) return GEMM_F16_ERR_INVALID_VALUE;
    in[nin++] = Span{x, e};
    if (!view_extent(D, E, stride_ri, stride_re, &e) || __builtin_mul_overflow(e, 2, &e)) return GEMM_F16_ERR_INVALID_VALUE;
    in[nin++] = Span{router, e};
    const moe_f16_weight* ws[3] = {gate, up, down};
    for (int i = 0; i < 3; ++i) {
        int64_t data, scales;
        if (!weight_span(*ws[i], E, i < 2 ? D : F, i < 2 ? F : D, &data, &scales)) return GEMM_F16_ERR_INVALID_VALUE;
        in[nin++] = Span{ws[i]->data, data};
        if (scales) in[nin++] = Span{ws[i]->scales, scales};
    }
    if (!view_extent(T, D, ldy, 1, &e) || __builtin_mul_overflow(e, 2, &e)) return GEMM_F16_ERR_INVALID_VALUE;
    out[nout++] = Span{y, e};
    out[nout++] = Span{weights, T * top_k * 4};
    out[nout++] = Span{ids, T * top_k * 4};
    out[nout++] = Span{workspace, l.bytes};
    for (int i = 0; i < nout; ++i) {
        for (int j = 0; j < nin; ++j)
            if (overlaps(out[i].p, out[i].bytes, in[j].p, in[j].bytes)) return GEMM_F16_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlaps(out[i].p, out[i].bytes, out[j].p, out[j].bytes)) return GEMM_F16_ERR_ALIAS;
    }
    if (workspace_bytes < static_cast<size_t>(l.bytes)) return GEMM_F16_ERR_OUT_OF_MEMORY;
    Device dev;
    gemm_f16_status st = current_device(&dev);
    if (st != GEMM_F16_OK) return st;
    for (int i = 0; i < nin; ++i)
        if (!device_range_ok(in[i].p, in[i].bytes)) return GEMM_F16_ERR_INVALID_VALUE;
    for (int i = 0; i < nout; ++i)
        if (!device_range_ok(out[i].p, out[i].bytes)) return GEMM_F16_ERR_INVALID_VALUE;

    moe_dev::Params p = {};
    p.x = static_cast<const __half*>(x);
    p.sxt = stride_xt, p.sxi = stride_xi;
    p.router = static_cast<const __half*>(router);
    p.sri = stride_ri, p.sre = stride_re;
    p.gate = weight_of(*gate, E, D, F);
    p.up = weight_of(*up, E, D, F);
    p.down = weight_of(*down, E, F, D);
    p.T = static_cast<int32_t>(T), p.D = static_cast<int32_t>(D), p.F = static_cast<int32_t>(F);
    p.E = static_cast<int32_t>(E), p.top = static_cast<int32_t>(top_k);
    p.renorm = renormalize != 0, p.act = act;
    p.dp = static_cast<int32_t>(l.dp), p.fp = static_cast<int32_t>(l.fp);
    p.y = static_cast<__half*>(y);
    p.ldy = ldy;
    p.weights = weights;
    p.ids = ids;
    uint8_t* base = static_cast<uint8_t*>(workspace);
    p.zero = reinterpret_cast<int*>(base);
    p.nzero = static_cast<int32_t>(kControlBytes / 4);
    p.ctl = reinterpret_cast<moe_dev::Control*>(base);
    p.counts = reinterpret_cast<int32_t*>(base + 256);
    if (gate->format == MOE_F16_WEIGHT_MXF4) {
        p.xq = base + l.xq;
        p.xs = base + l.xs;
        p.xq_pitch = static_cast<int32_t>(l.dq);
        p.xs_pitch = static_cast<int32_t>(l.dw);
    }
    p.parts = reinterpret_cast<float*>(base + l.parts);
    p.xp = reinterpret_cast<__half*>(base + l.xp);
    p.hp = reinterpret_cast<__half*>(base + l.hp);
    p.test_stall = option(GEMM_F16_OPT_TEST_STALL) == 1;
    p.timeout_ns = timeout_ns();
    p.status = dev.status;

    const bool aligned16 = aligned(router, 16);
    st = aligned16 && stride_ri == 1 && stride_re % 8 == 0   ? launch_route<moe_dev::kInContiguous>(p, stream)
         : aligned16 && stride_re == 1 && stride_ri % 8 == 0 ? launch_route<moe_dev::kOutContiguous>(p, stream)
                                                              : launch_route<moe_dev::kAnyStrides>(p, stream);
    if (st != GEMM_F16_OK) return st;
    if (gate->format == MOE_F16_WEIGHT_MXF4)
        return launch_stream<moe_dev::kStreamMxf4>(p, l, base, ws, dev.sms, stream);
    if (rows_aligned(*gate, E) && rows_aligned(*up, E) && rows_aligned(*down, E))
        return launch_stream<moe_dev::kStreamRows>(p, l, base, ws, dev.sms, stream);
    if (cols_aligned(*gate, E) && cols_aligned(*up, E) && cols_aligned(*down, E))
        return launch_stream<moe_dev::kStreamCols>(p, l, base, ws, dev.sms, stream);
    if (gate->stride_i == 1 && up->stride_i == 1 && down->stride_i == 1)
        return launch_experts<moe_dev::kF16Rows, 3>(p, dev.sms, stream);
    if (gate->stride_o == 1 && up->stride_o == 1 && down->stride_o == 1)
        return launch_experts<moe_dev::kF16Cols, 3>(p, dev.sms, stream);
    return launch_experts<moe_dev::kF16Strided, 3>(p, dev.sms, stream);
}

}  // extern "C"
