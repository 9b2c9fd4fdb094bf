// Host side of dcnv4_predictor_backward (declared in include/dcnv4.h).
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <map>
#include <mutex>

#include "dcnv4.h"
#include "dcnv4_internal.h"
#include "dcnv4_predictor_backward.cuh"

namespace {

#include "dcnv4_host_common.inl"

#include "dcnv4_unit_common.inl"

// Tiles, slices and walkers, from the sizes alone (and a nominal 148 SMs): what
// is left to choose the sums' order, and with it the result's bits, is dtype and
// which buffers TMA can take (launch()).
dcnv4::PredBwdParams make_params(int M, int C, int G, long long P, long long NO) {
    dcnv4::PredBwdParams p{};
    p.M = M; p.C = C; p.G = G; p.P = static_cast<int>(P); p.NO = static_cast<int>(NO);
    p.tiles = static_cast<int>((static_cast<long long>(M) + 127) / 128);
    p.chunks = (p.NO + 63) / 64;
    p.wrows = p.chunks * 64;
    p.wpitch = (C + 63) / 64 * 64;
    p.groups = (p.NO + 127) / 128;
    const long long per = static_cast<long long>(p.groups) * ((C + 127) / 128);
    // one walker, and so no launch to join partial sums, for one or two tiles. Measured from a graph, one walker
    // against several: 196 pixels x 256 fp16 channels x 432 slots 21.8 us against 23.7, x 512 x 864 23.6 against 43.9;
    // x 64 bf16 x 108 10.1 against 9.1, x 320 fp32 x 192 22.2 against 21.0 (less than the launch that the host is
    // spared). 257 pixels of the four: 26.9 against 24.1, 28.5 against 45.0, 12.6 against 9.3, 28.0 against 21.2.
    p.walkers = p.tiles <= 2 ? 1 : static_cast<int>(std::max<long long>(1, std::min<long long>(p.tiles, 148 / per)));
    return p;
}

int planes_of(int dtype) { return dtype == DCNV4_F32 ? 3 : dtype == DCNV4_F16 ? 2 : 1; }

// Workspace: W's planes, the walkers' partial sums of grad_weight, of grad_bias.
struct Layout {
    size_t part, pbias, bytes;
};
Layout layout(const dcnv4::PredBwdParams& p, int dtype) {
    Layout l{};
    auto up = [](size_t v) { return (v + 255) / 256 * 256; };
    l.part = up(static_cast<size_t>(planes_of(dtype)) * p.wrows * p.wpitch * 2);
    l.pbias = l.part + up(static_cast<size_t>(p.walkers) * p.NO * p.C * 4);
    l.bytes = p.M == 0 ? 0 : l.pbias + up(static_cast<size_t>(p.walkers) * p.NO * 4);
    return l;
}

bool tile_map(CUtensorMap* map, CUtensorMapDataType type, int e, void* base, long long cols, long long rows,
              long long planes, int box_cols, int box_rows) {
    auto encode = tensor_map_encoder();
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                                static_cast<cuuint64_t>(planes)};
    const cuuint64_t str[2] = {static_cast<cuuint64_t>(cols * e), static_cast<cuuint64_t>(cols * rows * e)};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows), 1u}, es[3] = {1u, 1u, 1u};
    return encode && encode(map, type, 3, base, dims, str, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int CT, int WP>
int launch_grad_y(const CUtensorMap& wmap, const CUtensorMap& gmap, const CUtensorMap& omap, const float* grec, float* gy,
                  dcnv4::PredBwdParams p, int nsm, bool raw, cudaStream_t s) {
    constexpr unsigned smem = dcnv4::GradYShape<CT, WP>::kSmem;
    static_assert(smem <= kTileSmemLimit, "the stages do not fit");
    auto kern = raw ? dcnv4::pred_grad_y_kernel<CT, WP, true> : dcnv4::pred_grad_y_kernel<CT, WP, false>;
    if (smem_limit_once(reinterpret_cast<const void*>(kern), static_cast<int>(smem)) != cudaSuccess)
        return DCNV4_ERR_LAUNCH;
    p.slices = (p.C + CT - 1) / CT;
    const long long items = static_cast<long long>(p.tiles) * p.slices;
    return launch_chained(kern, dim3(static_cast<unsigned>(std::min<long long>(items, nsm))), dcnv4::kGradYThreads, smem, s,
                          wmap, gmap, omap, grec, gy, p);
}

// More tiles of pixels per walker than the bias's sums take in fp32 (the first walker has the most).
bool long_sums(const dcnv4::PredBwdParams& p) { return (p.tiles + p.walkers - 1) / p.walkers > dcnv4::kBiasRun; }

template <typename T, bool RAW>
int launch_grad_w(const CUtensorMap& gmap, const CUtensorMap& ymap, const float* grec, const T* y, float* part,
                  float* pbias, dcnv4::PredBwdParams p, cudaStream_t s) {
    using S = dcnv4::GradWShape<T, RAW>;
    static_assert(S::smem(16384u) <= kTileSmemLimit && S::smem(32768u) <= kTileSmemLimit, "the stages do not fit");
    p.ystep = p.C > 64 ? 32768u : 16384u;
    p.raws = S::raws(p.ystep);
    const unsigned smem = S::smem(p.ystep);
    auto kern = long_sums(p) ? dcnv4::pred_grad_w_kernel<T, RAW, true> : dcnv4::pred_grad_w_kernel<T, RAW, false>;
    if (smem_limit_once(reinterpret_cast<const void*>(kern), static_cast<int>(std::max(S::smem(16384u), S::smem(32768u)))) !=
        cudaSuccess)
        return DCNV4_ERR_LAUNCH;
    p.slices = (p.C + 127) / 128;
    return launch_chained(kern, dim3(static_cast<unsigned>(p.walkers) * p.slices * p.groups), dcnv4::kGradWThreads, smem, s,
                          gmap, ymap, grec, y, part, pbias, p);
}

// One reading of g for everything, where the sums fit the tensor memory and the planes the shared memory.
template <typename T>
int launch_grad_both(const CUtensorMap& gmap, const CUtensorMap& ymap, const CUtensorMap& omap, const T* y, const T* w,
                     float* gy, float* part, float* pbias, const dcnv4::PredBwdParams& p, cudaStream_t s) {
    constexpr unsigned smem = dcnv4::GradBothShape<T>::kSmem;
    static_assert(smem <= kTileSmemLimit, "the stages do not fit");
    auto kern = long_sums(p) ? dcnv4::pred_grad_both_kernel<T, true> : dcnv4::pred_grad_both_kernel<T, false>;
    if (smem_limit_once(reinterpret_cast<const void*>(kern), static_cast<int>(smem)) != cudaSuccess) return DCNV4_ERR_LAUNCH;
    return launch_chained(kern, dim3(static_cast<unsigned>(p.walkers)), dcnv4::kGradYThreads, smem, s, gmap, ymap, omap, y, w,
                          gy, part, pbias, p);
}

int launch_join(const float* part, const float* pbias, float* gw, float* gb, const dcnv4::PredBwdParams& p, cudaStream_t s) {
    const long long n = (static_cast<long long>(p.NO) * p.C + (gb ? p.NO : 0) + 31) / 32;
    if (p.direct) return DCNV4_OK;
    return launch_chained(dcnv4::pred_grad_w_join_kernel, dim3(static_cast<unsigned>(std::min<long long>(n, 148 * 4))), 512, 0, s,
                          part, pbias, gw, gb, p);
}

template <typename T>
int launch(const void* y, const void* w, const float* grec, float* gy, float* gw, float* gb, unsigned char* ws,
           dcnv4::PredBwdParams p, int dtype, cudaStream_t s) {
    constexpr int WP = dcnv4::split_planes<T>(), E = sizeof(T);
    const int nsm = sm_count();
    if (nsm <= 0) return DCNV4_ERR_CUDA;
    const Layout l = layout(p, dtype);
    __nv_bfloat16* planes = reinterpret_cast<__nv_bfloat16*>(ws);
    p.direct = p.walkers == 1 && aligned(gw, 16) ? 1 : 0;
    float *part = p.direct ? gw : reinterpret_cast<float*>(ws + l.part);
    float *pbias = !gb || p.direct ? gb : reinterpret_cast<float*>(ws + l.pbias);
    // TMA wants rows of whole 16-byte units on 16-byte boundaries (200,704 pixels x 64 bf16 channels with 81 slots, read
    // directly, take 93 us, with 108 by TMA 41 in one pass or 71 in two)
    const bool raw_g = p.NO % 4 == 0 && aligned(grec, 16), raw_w = raw_g && p.C * E % 16 == 0 && aligned(y, 16);
    p.tma_out = p.C % 4 == 0 && aligned(gy, 16) ? 1 : 0;
    CUtensorMap wmap{}, gmap{}, ymap{}, omap{};
    if (!tile_map(&wmap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, planes, p.wpitch, p.wrows, WP, 64, 64) ||
        (raw_g && !tile_map(&gmap, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, const_cast<float*>(grec), p.NO, p.M, 1, 32, 128)) ||
        (raw_w && !tile_map(&ymap, tma_dtype<T>(), E, const_cast<void*>(y), p.C, p.M, 1, 128 / E, 128)) ||
        (p.tma_out && !tile_map(&omap, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, gy, p.C, p.M, 1, 32, 128)))
        return DCNV4_ERR_CUDA;
    // 200,704 pixels x 64 channels x 108 slots: bf16 40.9 us against 71.2 by the kernels below, fp16 59.4 against 87.3;
    // 196 pixels: 8.6 against 12.2, 9.8 against 14.1 (replayed from a graph)
    if constexpr (WP <= 2) {
        if (p.C <= 64 && p.NO <= 128 && (WP == 1 || p.NO > 64) && raw_w && p.tma_out && aligned(w, 16)) {
            const int rc = launch_grad_both<T>(gmap, ymap, omap, static_cast<const T*>(y), static_cast<const T*>(w), gy,
                                               part, pbias, p, s);
            return rc ? rc : launch_join(part, pbias, gw, gb, p, s);
        }
    }
    const long long pairs = static_cast<long long>(p.wrows) * p.wpitch / 2;
    int rc = launch_chained(dcnv4::pred_split_weight_kernel<T>, dim3(static_cast<unsigned>(std::min<long long>((pairs + 255) / 256, 148 * 8))),
                            256, 0, s, static_cast<const T*>(w), planes, p);
    if (rc) return rc;
    // 128 channels per tile halve the readings of g (129,032 pixels x 128 channels x 216 slots: bf16 92.7 us against
    // 117.3, fp16 139 against 152); with many slots (long chains of truncated additions) or three weight planes
    // (shared memory) 64 channels leave room for three accumulators of order 0
    if constexpr (WP <= 2) {
        if (p.C > 64 && p.NO <= 256) rc = launch_grad_y<128, WP>(wmap, gmap, omap, grec, gy, p, nsm, raw_g, s);
        else rc = launch_grad_y<64, WP>(wmap, gmap, omap, grec, gy, p, nsm, raw_g, s);
    } else {
        rc = launch_grad_y<64, WP>(wmap, gmap, omap, grec, gy, p, nsm, raw_g, s);
    }
    if (rc) return rc;
    rc = raw_w ? launch_grad_w<T, true>(gmap, ymap, grec, static_cast<const T*>(y), part, pbias, p, s)
               : launch_grad_w<T, false>(gmap, ymap, grec, static_cast<const T*>(y), part, pbias, p, s);
    if (rc) return rc;
    return launch_join(part, pbias, gw, gb, p, s);
}

}  // namespace

extern "C" {

int dcnv4_predictor_backward_workspace(int M, int C, int G, int K, unsigned flags, int dtype, size_t* bytes) {
    long long P = 0, NO = 0;
    const int rc = check_projection(M, C, G, K, flags, dtype, &P, &NO);
    if (rc) return rc;
    if (!bytes) return DCNV4_ERR_NULL;
    *bytes = layout(make_params(M, C, G, P, NO), dtype).bytes;
    return DCNV4_OK;
}

int dcnv4_predictor_backward(const void* y, const void* weight, const float* grad_offset_mask, float* grad_y,
                             float* grad_weight, float* grad_bias, void* workspace, size_t workspace_size,
                             int M, int C, int G, int K, unsigned flags, int dtype, void* stream) {
    long long P = 0, NO = 0;
    const int rc = check_projection(M, C, G, K, flags, dtype, &P, &NO);
    if (rc) return rc;
    dcnv4::PredBwdParams p = make_params(M, C, G, P, NO);
    const int e = elem_size(dtype);
    const long long ny = static_cast<long long>(M) * C, nw = NO * C, nrec = M * NO;
    const long long need = static_cast<long long>(layout(p, dtype).bytes);
    // without pixels the weight's gradients are still written (zeros)
    if (!grad_weight || (M > 0 && (!y || !weight || !grad_offset_mask || !grad_y || !workspace))) return DCNV4_ERR_NULL;
    if (!aligned(y, e) || !aligned(weight, e) || !aligned(grad_offset_mask, 4) || !aligned(grad_y, 4) ||
        !aligned(grad_weight, 4) || !aligned(grad_bias, 4) || (M > 0 && !aligned(workspace, 256)))
        return DCNV4_ERR_ALIGN;
    if (M > 0 && workspace_size < static_cast<size_t>(need)) return DCNV4_ERR_WORKSPACE;
    const void* in[3] = {y, weight, grad_offset_mask};
    const long long in_bytes[3] = {ny * e, M > 0 ? nw * e : 0, nrec * 4};
    const void* out[4] = {grad_y, grad_weight, grad_bias, workspace};
    const long long out_bytes[4] = {ny * 4, nw * 4, grad_bias ? NO * 4 : 0, M > 0 ? need : 0};
    for (int o = 0; o < 4; ++o) {
        for (int i = 0; i < 3; ++i)
            if (overlap(out[o], out_bytes[o], in[i], in_bytes[i])) return DCNV4_ERR_ALIAS;
        for (int q = 0; q < o; ++q)
            if (overlap(out[o], out_bytes[o], out[q], out_bytes[q])) return DCNV4_ERR_ALIAS;
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (M == 0) {
        if (cudaMemsetAsync(grad_weight, 0, static_cast<size_t>(nw) * 4, s) != cudaSuccess) return DCNV4_ERR_CUDA;
        if (grad_bias && cudaMemsetAsync(grad_bias, 0, static_cast<size_t>(NO) * 4, s) != cudaSuccess)
            return DCNV4_ERR_CUDA;
        return DCNV4_OK;
    }
    p.status = dcnv4_host::device_status_word();
    if (!p.status) return DCNV4_ERR_CUDA;
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    switch (dtype) {
        case DCNV4_F32: return launch<float>(y, weight, grad_offset_mask, grad_y, grad_weight, grad_bias, ws, p, dtype, s);
        case DCNV4_F16: return launch<__half>(y, weight, grad_offset_mask, grad_y, grad_weight, grad_bias, ws, p, dtype, s);
        default: return launch<__nv_bfloat16>(y, weight, grad_offset_mask, grad_y, grad_weight, grad_bias, ws, p, dtype, s);
    }
}

}  // extern "C"
